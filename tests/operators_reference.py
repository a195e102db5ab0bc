"""Plain 64-bit forms of the operators around the GEMMs, for the GPU tests: loops and numpy, written
from the definitions in include/fp8gemm.h."""
from __future__ import annotations

import numpy as np


def route(logits, k, mask=None, renormalize=True):
    """logits float64 [S, T, E] -> dict of ids, weights, counts, loss, slope and p (rows not routed: 0)."""
    S, T, E = logits.shape
    ids = np.full((S, T, k), -1, np.int32)
    weights, p = np.zeros((S, T, k)), np.zeros((S, T, E))
    counts, loss, slope = np.zeros((S, E), np.int32), np.zeros(S), np.zeros((S, E))
    for s in range(S):
        routed = 0
        for t in range(T):
            row = logits[s, t]
            if (mask is not None and not mask[s, t]) or not np.any(row > -np.inf):
                continue
            routed += 1
            order = sorted((e for e in range(E) if row[e] > -np.inf), key=lambda e: (-row[e], e))[:k]
            p[s, t] = np.exp(row - row[order[0]])
            p[s, t] /= p[s, t].sum()
            picked = p[s, t][order]
            ids[s, t, :len(order)] = order
            weights[s, t, :len(order)] = picked / picked.sum() if renormalize else picked
            counts[s, order] += 1
        if routed:
            slope[s] = E * counts[s] / counts[s].sum() / routed
            loss[s] = (slope[s] * p[s].sum(0)).sum()
    return dict(ids=ids, weights=weights, counts=counts, loss=loss, slope=slope, p=p)


def route_backward(fwd, grad_weights, grad_loss, renormalize=True):
    """(gradient, bound): the gradient of the logits, and the sums of absolute terms behind each value,
    which rounding errors are proportional to."""
    ids, p, slope = fwd["ids"], fwd["p"], fwd["slope"]
    S, T, E = p.shape
    grad, bound = np.zeros((S, T, E)), np.zeros((S, T, E))
    for s in range(S):
        for t in range(T):
            chosen = ids[s, t][ids[s, t] >= 0]
            if not chosen.size:
                continue
            h = grad_loss[s] * slope[s].copy() if grad_loss is not None else np.zeros(E)
            g = grad_weights[s, t][:chosen.size] if grad_weights is not None else np.zeros(chosen.size)
            if not renormalize:
                h[chosen] += g
            q = p[s, t]
            grad[s, t] = q * (h - (q * h).sum())
            bound[s, t] = q * (np.abs(h) + (q * np.abs(h)).sum())
            if renormalize:
                w = q[chosen] / q[chosen].sum()
                grad[s, t][chosen] += w * (g - (w * g).sum())
                bound[s, t][chosen] += w * (np.abs(g) + (w * np.abs(g)).sum())
    return grad, bound


def layout(ids, E, mmax=None, align=128):
    """(rows, m_indices of the occupied blocks) of the contiguous layout; (rows, masked_m) with mmax."""
    flat = ids.reshape(-1)
    counts = [int((flat == e).sum()) for e in range(E)]
    starts, at = [], 0
    for e in range(E):
        starts.append(e * mmax if mmax else at)
        at += -(-counts[e] // align) * align
    rows, seen = np.full(flat.shape, -1, np.int32), [0] * E
    for i, e in enumerate(flat):
        if 0 <= e < E:
            if not mmax or seen[e] < mmax:
                rows[i] = starts[e] + seen[e]
            seen[e] += 1
    if mmax:
        return rows.reshape(ids.shape), np.minimum(counts, mmax).astype(np.int32)
    group = np.full(at, -1, np.int32)
    for e in range(E):
        group[starts[e]:starts[e] + counts[e]] = e
    return rows.reshape(ids.shape), group


def combine(C, rows, weights):
    """(out, sums of |w C|) with C float64 [M, N]."""
    out, size = np.zeros((rows.shape[0], C.shape[1])), np.zeros((rows.shape[0], C.shape[1]))
    for t in range(rows.shape[0]):
        for j, r in enumerate(rows[t]):
            if r >= 0:
                w = 1.0 if weights is None else weights[t, j]
                out[t] += w * C[r]
                size[t] += np.abs(w * C[r])
    return out, size


def lora(C, x, a, b, adapters, scaling):
    """(out, |h| sums, |delta| sums): with h = A x, the sums of |A| |x| carried through |B|, and of
    |s h| |B|."""
    out, size_h, size_d = C.copy(), np.zeros(C.shape), np.zeros(C.shape)
    for m, i in enumerate(adapters):
        if 0 <= i < a.shape[0]:
            s = 1.0 if scaling is None else scaling[i]
            h = a[i] @ x[m]
            out[m] += s * (b[i] @ h)
            size_h[m] = abs(s) * (np.abs(b[i]) @ (np.abs(a[i]) @ np.abs(x[m])))
            size_d[m] = abs(s) * (np.abs(b[i]) @ np.abs(h))
    return out, size_h, size_d

"""GPU tests of the operators around the GEMMs against plain 64-bit forms: the router with its balance
loss and gradient, the experts' row layouts, the cast into them, the weighted sum and its gradients,
the low-rank adapters; then all of them in a row, captured graphs, streams and long offsets.

Tolerances are sums of the roundings that a value passes through, u = 2^-24 for each in fp32 and
eps / 2 for the last one to the output's type:
  softmax terms   e^(x - m): the difference and the product with log2(e) each round an argument of
                  size d, so 2 d u relative, plus 2 ulp of exp2f; the sum over E adds (values per
                  lane + lanes) u, at most 38 u; the division u
  sums of n terms n u times the sum of the terms' sizes, in any order
  tensor cores    products are exact; each accumulation is taken to lose up to 2 u of the sum of sizes
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
from tests import operators_reference as ref

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF16 = 2.0 ** -8  # half a step
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module")
def fg():
    import moe_grouped_gemm_08_b200 as lib
    torch.cuda.set_device(0)
    lib.init(0)
    return lib


def f64(t):
    return t.detach().double().cpu().numpy()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rel_softmax(logits):
    """Relative error allowed for a softmax value of these (finite) logits."""
    finite = logits[np.isfinite(logits)]
    d = float(finite.max() - finite.min()) if finite.size else 0.0
    return (2 * min(d, 110.0) + 50) * U


# ------------------------------------------------------------------------------------- the router
ROUTES = [  # S, T, E, k, dtype
    (1, 1, 1, 1, "fp32"), (1, 1, 256, 8, "bf16"), (1, 2, 5, 5, "fp16"), (2, 3, 8, 2, "fp16"), (3, 77, 60, 4, "fp16"),
    (1, 300, 64, 6, "bf16"), (2, 65, 96, 6, "fp32"), (1, 515, 128, 1, "bf16"), (1, 700, 256, 8, "fp32"),
    (2, 129, 255, 10, "bf16"), (1, 40, 512, 16, "fp16"), (1, 33, 1024, 32, "fp32"), (1, 9, 1000, 32, "bf16"),
    (1, 5, 33, 32, "fp32"),
]


def route_case(S, T, E, k, dtype, masked, closed, seed=0):
    g = gen(1000 * S + 10 * T + E + seed)
    logits = 2 * torch.randn(S, T, E, generator=g)
    if closed:
        logits = logits.masked_fill(torch.rand(S, T, E, generator=g) < 0.4, -np.inf)
        logits[:, T // 2] = -np.inf  # a row whose mask leaves nothing
        logits[:, T - 1] = torch.finfo(DTYPES[dtype]).min  # and one of the type's lowest value
    logits = logits.to(DTYPES[dtype])
    mask = None
    if masked:
        mask = torch.rand(S, T, generator=g) < 0.7
        mask[0] = False if S > 1 else mask[0]  # a sequence without tokens
        junk = torch.tensor([np.nan, np.inf, torch.finfo(logits.dtype).min, -np.inf]).to(logits.dtype)
        logits = torch.where(mask[..., None], logits, junk[torch.arange(E) % 4])
    return logits, mask


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("masked,closed", [(False, False), (True, False), (True, True)])
@pytest.mark.parametrize("S,T,E,k,dtype", ROUTES)
def test_route_and_its_gradient(fg, S, T, E, k, dtype, masked, closed, renorm):
    logits, mask = route_case(S, T, E, k, dtype, masked, closed)
    want = ref.route(f64(logits), k, None if mask is None else mask.numpy(), renorm)
    dev = logits.cuda()
    ids, weights, counts, loss, slope = fg.moe_route(dev, k, mask=None if mask is None else mask.cuda(),
                                                     renormalize=renorm)
    assert np.array_equal(ids.cpu().numpy(), want["ids"])
    assert np.array_equal(counts.cpu().numpy(), want["counts"])
    live = want["ids"][..., 0] >= 0
    rel = rel_softmax(f64(logits)[live]) if live.any() else U
    assert np.all(np.abs(f64(weights) - want["weights"]) <= 2 * rel * want["weights"] + 2.0 ** -126)
    assert np.all(np.abs(f64(slope) - want["slope"]) <= 4 * U * want["slope"])
    assert np.all(np.abs(f64(loss) - want["loss"]) <= (rel + (T + E + 8) * U) * want["loss"])
    g = gen(7)
    gw, gl = torch.randn(S, T, k, generator=g), torch.randn(S, generator=g) * T
    for use_w, use_l in ((True, True), (True, False), (False, True), (False, False)):
        got = fg.moe_route_backward(dev, ids, slope, gw.cuda() if use_w else None, gl.cuda() if use_l else None,
                                    renormalize=renorm)
        grad, size = ref.route_backward(want, f64(gw) if use_w else None, f64(gl) if use_l else None, renorm)
        assert got.dtype == logits.dtype
        half = torch.finfo(logits.dtype).eps / 2
        least = torch.finfo(logits.dtype).smallest_normal * 2 * half
        # p, h and the sum of p h each carry rel, at most 70 additions behind a value
        tol = (4 * rel + 80 * U) * size * (1 + half) + half * np.abs(grad) + least
        assert np.all(np.abs(f64(got) - grad) <= tol), np.max(np.abs(f64(got) - grad) - tol)


def test_route_ties_take_the_lowest_expert(fg):
    logits = torch.randint(-2, 3, (300, 200), generator=gen(3)).float()
    logits[0] = 0.0
    logits[1, ::2], logits[1, 1::2] = 0.0, -0.0  # equal
    for dtype in DTYPES.values():
        ids, _, counts, _, _ = fg.moe_route(logits.to(dtype).cuda(), 9)
        want = ref.route(f64(logits)[None], 9)
        assert np.array_equal(ids.cpu().numpy(), want["ids"][0])
        assert np.array_equal(counts.cpu().numpy(), want["counts"][0])


def test_route_nan_and_infinity(fg):
    logits = torch.randn(4, 16, generator=gen(4))
    logits[0, 3] = np.nan
    logits[1, :] = np.nan
    logits[2, 5] = np.inf
    ids, weights, counts, loss, _ = fg.moe_route(logits.cuda(), 4)
    ids = ids.cpu().numpy()
    assert 3 not in ids[0] and (ids[1] == -1).all() and ids[2, 0] == 5
    assert all(len(set(r)) == 4 for r in ids[[0, 2, 3]])
    assert counts.sum().item() == 12 and torch.isnan(loss).item()
    assert torch.isfinite(weights[3]).all() and (weights[1] == 0).all()


def test_route_without_tokens(fg):
    ids, weights, counts, loss, slope = fg.moe_route(torch.empty(2, 0, 8, device="cuda"), 3)
    assert ids.shape == weights.shape == (2, 0, 3)
    assert (counts == 0).all() and (loss == 0).all() and (slope == 0).all()
    assert fg.moe_route_backward(torch.empty(2, 0, 8, device="cuda"), ids, slope, weights, loss).shape == (2, 0, 8)
    assert fg.moe_route(torch.empty(0, 5, 8, device="cuda"), 3)[0].shape == (0, 5, 3)


def test_route_repeats_bit_for_bit(fg):
    logits = torch.randn(3, 5000, 256, generator=gen(5)).cuda()
    first = fg.moe_route(logits, 8)
    for _ in range(5):
        for a, b in zip(first, fg.moe_route(logits, 8)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("renorm", [True, False])
def test_route_gradient_against_differences(fg, renorm):
    """Central differences of the 64-bit loss sum(gw * weights) + sum(gl * loss), with the choices held
    (a step of 1e-4 leaves gaps of 0.01 between the logits in order); the truncation is below
    step^2 times the third derivative, at most 6 times the sum of the terms' sizes."""
    S, T, E, k, step = 2, 5, 7, 3, 1e-4
    g = gen(6)
    logits = (torch.stack([torch.randperm(E * 40, generator=g)[:E] for _ in range(S * T)]).float() / 100).view(S, T, E)
    gw, gl = torch.randn(S, T, k, generator=g), torch.randn(S, generator=g) * T
    ids, _, _, _, slope = fg.moe_route(logits.cuda(), k, renormalize=renorm)
    got = f64(fg.moe_route_backward(logits.cuda(), ids, slope, gw.cuda(), gl.cuda(), renormalize=renorm))
    base = ref.route(f64(logits), k, None, renorm)
    size = ref.route_backward(base, f64(gw), f64(gl), renorm)[1]

    def value(l):
        r = ref.route(l, k, None, renorm)
        assert np.array_equal(r["ids"], base["ids"])
        return (f64(gw) * r["weights"]).sum() + (f64(gl) * r["loss"]).sum()

    for s in range(S):
        for t in range(T):
            for e in range(E):
                up, down = f64(logits), f64(logits)
                up[s, t, e] += step
                down[s, t, e] -= step
                want = (value(up) - value(down)) / (2 * step)
                assert abs(got[s, t, e] - want) <= (6 * step ** 2 + 200 * U) * size[s, t, e] + 1e-10


# ------------------------------------------------------------------------------------- layouts
def choices(T, k, E, total, seed, none=0.0):
    g = gen(seed)
    ids = torch.stack([torch.randperm(total, generator=g)[:k] for _ in range(T)]).to(torch.int32).view(T, k)
    ids = torch.where(torch.rand(T, k, generator=g) < none, -1, ids)
    return ids


LAYOUTS = [(1, 1, 1, 1), (1, 8, 256, 256), (7, 3, 5, 5), (64, 8, 32, 256), (300, 2, 3, 3), (2048, 1, 7, 7),
           (2049, 1, 7, 7), (3000, 8, 64, 64), (777, 32, 1024, 1024), (5000, 4, 4, 9)]


@pytest.mark.parametrize("T,k,E,total", LAYOUTS)
def test_layouts(fg, T, k, E, total):
    for none in (0.0, 0.3, 1.0):
        ids = choices(T, k, E, total, T + E, none)
        if none == 0.3:
            ids[0, 0], ids[-1, -1] = 2 ** 31 - 1, -(2 ** 31)  # any value outside [0, E)
            ids[T // 2] = 0  # the same expert in every choice of a token
        rows, group = fg.moe_layout_contiguous(ids.cuda(), E)
        want_rows, want_group = ref.layout(ids.numpy(), E)
        assert np.array_equal(rows.cpu().numpy(), want_rows)
        group = group.cpu().numpy()
        assert group.size == fg.moe_layout_rows(T * k, E) >= want_group.size
        assert np.array_equal(group[:want_group.size], want_group) and (group[want_group.size:] == -1).all()
        for mmax in (1, max(1, T // 4), T * k):
            rows, masked_m = fg.moe_layout_masked(ids.cuda(), E, mmax)
            want_rows, want_m = ref.layout(ids.numpy(), E, mmax)
            assert np.array_equal(rows.cpu().numpy(), want_rows)
            assert np.array_equal(masked_m.cpu().numpy(), want_m)


@pytest.mark.parametrize("pairs,E", [(80_000, 256), (1_200_000, 1000), (300_000, 3)])
def test_layouts_of_many_pairs(fg, pairs, E):
    ids = torch.randint(-1, E + 1, (pairs, 1), generator=gen(pairs)).to(torch.int32)
    flat = ids.flatten().numpy()
    live = (flat >= 0) & (flat < E)
    order = np.argsort(np.where(live, flat, E), kind="stable")
    counts = np.bincount(flat[live], minlength=E)
    place = np.empty(pairs, np.int64)
    place[order] = np.arange(pairs)
    place -= np.concatenate([[0], np.cumsum(counts)])[np.where(live, flat, E)]
    padded = -(-counts // 128) * 128
    start = np.cumsum(padded) - padded
    rows, group = fg.moe_layout_contiguous(ids.cuda(), E)
    assert np.array_equal(rows.cpu().numpy()[:, 0], np.where(live, start[np.clip(flat, 0, E - 1)] + place, -1))
    want = np.full(group.numel(), -1, np.int32)
    for e in range(E):
        want[start[e]:start[e] + counts[e]] = e
    assert np.array_equal(group.cpu().numpy(), want)
    mmax = int(counts.max()) - 5
    rows, masked_m = fg.moe_layout_masked(ids.cuda(), E, mmax)
    assert np.array_equal(rows.cpu().numpy()[:, 0], np.where(live & (place < mmax), flat * mmax + place, -1))
    assert np.array_equal(masked_m.cpu().numpy(), np.minimum(counts, mmax))


def test_layout_without_pairs(fg):
    empty = torch.empty(0, 4, dtype=torch.int32, device="cuda")
    rows, group = fg.moe_layout_contiguous(empty, 8)
    assert rows.shape == (0, 4) and group.numel() == 0
    rows, masked_m = fg.moe_layout_masked(empty, 8, 16)
    assert rows.shape == (0, 4) and (masked_m == 0).all()


# ------------------------------------------------------------------------------------- dispatch
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("T,k,E,K,mmax", [(1, 1, 1, 16, 0), (5, 2, 3, 128, 0), (33, 3, 4, 2064, 0), (130, 8, 16, 1040, 0),
                                          (64, 4, 8, 7168, 24), (9, 32, 40, 272, 9)])
def test_dispatch_stores_the_cast_rows(fg, T, k, E, K, mmax, fmt):
    g = gen(T + K)
    x = (torch.randn(T, K, generator=g) * 10.0 ** torch.empty(T, 1).uniform_(-3, 3, generator=g)).to(torch.bfloat16)
    x[0, :min(K, 128)] = 0  # an all-zero block
    ids = choices(T, k, E, max(E, k), T, 0.1).cuda()
    q, s = fg.cast_fp8_rows(x.cuda(), fmt=fmt)
    q, s = q.cpu(), s.cpu()
    KB = -(-K // 128)
    if mmax:
        rows, _ = fg.moe_layout_masked(ids, E, mmax)
        shape, scales = (E, mmax), (E, KB, fg.sfa_ld(mmax))
    else:
        rows, group = fg.moe_layout_contiguous(ids, E)
        shape, scales = (group.numel(),), (KB, fg.sfa_ld(group.numel()))
    A = torch.full(shape + (K,), 0xA5, dtype=torch.uint8, device="cuda")
    sfa = torch.full(scales, -7.0, device="cuda")
    fg.moe_dispatch_fp8(x.cuda(), rows, A=A, sfa=sfa, fmt=fmt)
    want_A = torch.full(shape + (K,), 0xA5, dtype=torch.uint8).view(-1, K)
    want_s = torch.full(scales, -7.0)
    for t in range(T):
        for r in rows[t].tolist():
            if r >= 0:
                want_A[r] = q[t]
                (want_s[r // mmax] if mmax else want_s)[:, r % mmax if mmax else r] = s[:, t]
    assert torch.equal(A.cpu().view(-1, K), want_A)  # rows that no choice has are left as they were
    assert torch.equal(sfa.cpu(), want_s)
    A2, sfa2 = fg.moe_dispatch_fp8(x.cuda(), rows, shape=shape, fmt=fmt)
    held = rows[rows >= 0].long()
    assert torch.equal(A2.view(-1, K)[held], A.view(-1, K)[held])
    assert sfa2.shape == sfa.shape


# ------------------------------------------------------------------------------------- combine
@pytest.mark.parametrize("T,k,E,N,mmax", [(1, 1, 1, 8, 0), (5, 2, 3, 136, 0), (33, 3, 4, 2056, 0), (130, 8, 16, 264, 0),
                                          (64, 4, 8, 7168, 24), (9, 32, 40, 512, 9), (3, 9, 9, 4104, 0)])
def test_combine_and_its_gradients(fg, T, k, E, N, mmax):
    g = gen(T + N)
    ids = choices(T, k, E, max(E, k), T, 0.2)
    ids[T // 2] = -1  # a token without rows
    rows, group = (fg.moe_layout_masked(ids.cuda(), E, mmax) if mmax else fg.moe_layout_contiguous(ids.cuda(), E))
    M = E * mmax if mmax else group.numel()
    C = torch.randn(M, N, generator=g).to(torch.bfloat16)
    rows_h = rows.cpu().numpy()
    unused = np.setdiff1d(np.arange(M), rows_h[rows_h >= 0])
    C[unused] = float("nan")  # rows of no choice are not read
    weights = torch.randn(T, k, generator=g)
    dev = C.cuda().view(E, mmax, N) if mmax else C.cuda()
    C64 = np.nan_to_num(f64(C))
    for w in (weights, None):
        out = fg.moe_combine(dev, rows, None if w is None else w.cuda())
        want, size = ref.combine(C64, rows_h, None if w is None else f64(w))
        assert np.all(np.abs(f64(out) - want) <= (k + 1) * U * size * (1 + BF16) + BF16 * np.abs(want) + 1e-40)
        assert (out[T // 2] == 0).all()
    go = torch.randn(T, N, generator=g).to(torch.bfloat16)
    keep = torch.full(dev.shape, 3.0, dtype=torch.bfloat16, device="cuda")
    grad_C, grad_w = fg.moe_combine_backward(go.cuda(), dev, rows, weights.cuda(), grad_C=keep)
    assert grad_C is keep
    want_C, want_w, size_w = np.full((M, N), 3.0), np.zeros((T, k)), np.zeros((T, k))
    for t in range(T):
        for j, r in enumerate(rows_h[t]):
            if r >= 0:
                want_C[r] = float(weights[t, j]) * f64(go[t])
                want_w[t, j] = f64(go[t]) @ C64[r]
                size_w[t, j] = np.abs(f64(go[t])) @ np.abs(C64[r])
    assert np.all(np.abs(f64(grad_C).reshape(M, N) - want_C) <= (BF16 + 2 * U) * np.abs(want_C))
    assert np.all(np.abs(f64(grad_w) - want_w) <= (N / 8 + 40) * U * size_w)


def test_combine_gradient_of_pairs_without_a_row_is_zero(fg):
    """... whatever the gradient of the sum and the weights hold."""
    rows = torch.tensor([[-1, 0, -1], [1, -1, -1]], dtype=torch.int32, device="cuda")
    C = torch.ones(2, 24, dtype=torch.bfloat16, device="cuda")
    go = torch.full((2, 24), float("inf"), dtype=torch.bfloat16, device="cuda")
    go[1] = float("nan")
    w = torch.where(rows < 0, float("nan"), 1.0)
    grad_w = fg.moe_combine_backward(go, C, rows, w)[1]
    assert (grad_w[rows < 0] == 0).all() and torch.isinf(grad_w[0, 1]) and torch.isnan(grad_w[1, 0])
    assert (fg.moe_combine(C, rows, w) == 1).all()


def test_combine_rows_out_of_range_are_none(fg):
    C = torch.ones(4, 16, dtype=torch.bfloat16, device="cuda")
    rows = torch.tensor([[0, 4, -5], [2 ** 31 - 1, 3, 2]], dtype=torch.int32, device="cuda")
    assert fg.moe_combine(C, rows).float()[:, 0].tolist() == [1.0, 2.0]
    grad_C, grad_w = fg.moe_combine_backward(C[:2].contiguous(), C, rows, torch.ones(2, 3, device="cuda"))
    assert grad_w.tolist() == [[16.0, 0.0, 0.0], [0.0, 16.0, 16.0]]
    A, sfa = fg.moe_dispatch_fp8(C[:2].contiguous(), rows, A=torch.zeros(4, 16, dtype=torch.uint8, device="cuda"),
                                 sfa=torch.zeros(1, 4, device="cuda"))
    assert (A.sum(1) > 0).tolist() == [True, False, True, True]


# ------------------------------------------------------------------------------------- adapters
LORAS = [  # M, K, N, R, L
    (1, 16, 8, 8, 1), (1, 7168, 4096, 16, 4), (3, 48, 40, 24, 2), (17, 272, 264, 16, 1), (40, 528, 72, 32, 3),
    (64, 1040, 1032, 40, 64), (130, 256, 520, 64, 5), (33, 512, 136, 128, 2), (300, 144, 104, 96, 4),
    (700, 400, 200, 8, 3), (500, 272, 136, 128, 2), (1000, 1040, 264, 64, 5), (2100, 80, 72, 32, 300), (257, 16, 8, 48, 1),
    (1500, 4112, 520, 40, 9), (600, 64, 40, 8, 1500), (256, 528, 264, 128, 30), (255, 144, 72, 72, 1),
]


def lora_case(M, K, N, R, L, seed=0):
    g = gen(M + K + N + seed)
    adapters = torch.randint(-1, L + 1, (M,), generator=g).to(torch.int32)  # L and -1: none
    if M > 2:
        adapters[1] = 2 ** 31 - 1
        adapters[2] = -(2 ** 31)
    else:
        adapters[:] = L - 1
    return dict(C=torch.randn(M, N, generator=g).to(torch.bfloat16), x=torch.randn(M, K, generator=g).to(torch.bfloat16),
                lora_a=(torch.randn(L, R, K, generator=g) / K ** 0.5).to(torch.bfloat16),
                lora_b=torch.randn(L, N, R, generator=g).to(torch.bfloat16), adapters=adapters,
                scaling=torch.randn(L, generator=g))


def lora_check(got, case, K, R, scaling=True):
    want, size_h, size_d = ref.lora(*(f64(case[n]) for n in ("C", "x", "lora_a", "lora_b")), case["adapters"].numpy(),
                                    f64(case["scaling"]) if scaling else None)
    # h: K products and the sums of the parts; its 16 bits (2^-16); the second product twice over R
    tol = (2 * (K / 16 + 40)) * U * size_h + (2.0 ** -16 + 2 * (R / 4 + 8) * U) * size_d
    tol = tol * (1 + BF16) + BF16 * np.abs(want)
    err = np.abs(f64(got) - want)
    assert np.all(err <= tol), (np.max(err - tol), np.argwhere(err > tol)[:4])
    none = (case["adapters"] < 0) | (case["adapters"] >= case["lora_a"].shape[0])
    assert torch.equal(got.cpu()[none], case["C"][none])  # bit for bit


@pytest.mark.parametrize("M,K,N,R,L", LORAS)
def test_lora_add(fg, M, K, N, R, L):
    case = lora_case(M, K, N, R, L)
    dev = {n: t.cuda() for n, t in case.items()}
    out = torch.full((M, N), -1.0, dtype=torch.bfloat16, device="cuda")
    assert fg.lora_add(**dev, out=out) is out
    lora_check(out, case, K, R)
    assert torch.equal(dev["C"].cpu(), case["C"])
    assert torch.equal(fg.lora_add(**dev), out)
    lora_check(fg.lora_add(**{**dev, "scaling": None}), case, K, R, scaling=False)
    assert torch.equal(fg.lora_add(**dev, out=dev["C"]), out)  # in place
    assert fg.lora_status() == 0


@pytest.mark.parametrize("M", [5, 600])
def test_lora_all_rows_of_one_adapter_or_none(fg, M):
    K, N, R, L = 320, 296, 16, 3
    case = lora_case(M, K, N, R, L)
    for fill in (1, -1):
        case["adapters"][:] = fill
        lora_check(fg.lora_add(**{n: t.cuda() for n, t in case.items()}), case, K, R)


def test_lora_rows_do_not_mix(fg):
    """A row's NaN and infinities stay in its row; a row of one adapter equals the row alone."""
    M, K, N, R, L = 50, 512, 256, 16, 2
    case = lora_case(M, K, N, R, L)
    case["adapters"][:] = torch.arange(M) % 2
    clean = fg.lora_add(**{n: t.cuda() for n, t in case.items()})
    case["x"][7] = float("nan")
    case["x"][8] = float("inf")
    got = fg.lora_add(**{n: t.cuda() for n, t in case.items()})
    keep = [m for m in range(M) if m not in (7, 8)]
    assert torch.equal(got[keep], clean[keep])
    assert torch.isnan(got[7]).all() and not torch.isfinite(got[8]).any()


def test_lora_empty(fg):
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    assert fg.lora_add(z(0, 8), z(0, 16), z(2, 8, 16), z(2, 8, 8), none).shape == (0, 8)
    C = torch.randn(3, 8, device="cuda").to(torch.bfloat16)
    ids = torch.zeros(3, dtype=torch.int32, device="cuda")
    assert torch.equal(fg.lora_add(C, z(3, 16), z(0, 8, 16), z(0, 8, 8), ids), C)  # no adapters at all
    assert torch.equal(fg.lora_add(C, z(3, 16), z(2, 0, 16), z(2, 8, 0), ids), C)  # rank 0
    big = torch.randn(100_000, 8, device="cuda").to(torch.bfloat16)
    ids = torch.zeros(100_000, dtype=torch.int32, device="cuda")
    assert torch.equal(fg.lora_add(big, z(100_000, 16), z(0, 8, 16), z(0, 8, 8), ids), big)


# ------------------------------------------------------------------------------------- refusals
def test_binding_refuses(fg):
    """Shapes, types, devices, streams and overlapping outputs, before anything is launched."""
    b = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    i = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    f = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    logits = f(4, 8)
    for bad in (0, 9):
        with pytest.raises(ValueError, match="top_k"):
            fg.moe_route(logits, bad)
    with pytest.raises(fg.FP8GemmError, match="UNSUPPORTED"):
        fg.moe_route(f(2, 64), 33)
    with pytest.raises(fg.FP8GemmError, match="UNSUPPORTED"):
        fg.moe_route(f(2, 1025), 2)
    with pytest.raises(ValueError, match="contiguous"):
        fg.moe_route(f(8, 4).t(), 2)
    with pytest.raises(TypeError, match="mask"):
        fg.moe_route(logits, 2, mask=torch.ones(4, device="cuda"))
    with pytest.raises(TypeError, match="mask"):
        fg.moe_route(logits, 2, mask=torch.ones(4, dtype=torch.bool))
    with pytest.raises(ValueError, match="mask must have shape"):
        fg.moe_route(logits, 2, mask=torch.ones(5, dtype=torch.bool, device="cuda"))
    with pytest.raises(ValueError, match="slope"):
        fg.moe_route_backward(logits, i(4, 2), f(7))
    with pytest.raises(ValueError, match="ids"):
        fg.moe_route_backward(logits, i(5, 2), f(8))
    with pytest.raises(ValueError, match="num_experts"):
        fg.moe_layout_contiguous(i(4, 2), 1025)
    with pytest.raises(ValueError, match="num_experts"):
        fg.moe_layout_masked(i(4, 2), 0, 4)
    with pytest.raises(ValueError, match="rows"):
        fg.moe_dispatch_fp8(b(4, 16), i(5, 2), shape=128)
    with pytest.raises(ValueError, match="shape"):
        fg.moe_dispatch_fp8(b(4, 16), i(4, 2))
    with pytest.raises(fg.FP8GemmError, match="ALIGNMENT"):
        fg.moe_dispatch_fp8(b(4, 24), i(4, 2), shape=128)
    with pytest.raises(ValueError, match="sfa must have shape"):
        fg.moe_dispatch_fp8(b(4, 16), i(4, 2), A=torch.zeros(128, 16, dtype=torch.uint8, device="cuda"), sfa=f(1, 127))
    C = b(12, 16)
    with pytest.raises(ValueError, match="out must not overlap C"):
        fg.moe_combine(C, i(4, 2), out=C[8:])
    with pytest.raises(ValueError, match="grad_C must not overlap C"):
        fg.moe_combine_backward(b(4, 16), C, i(4, 2), f(4, 2), grad_C=C)
    with pytest.raises(fg.FP8GemmError, match="UNSUPPORTED"):
        fg.moe_combine(C, i(4, 33))
    big = b(8, 16)
    with pytest.raises(ValueError, match="out must not overlap C"):
        fg.lora_add(big[:4], b(4, 16), b(1, 8, 16), b(1, 16, 8), i(4), out=big[2:6])
    with pytest.raises(ValueError, match="out must not overlap x"):
        fg.lora_add(C[:4], big[:4], b(1, 8, 16), b(1, 16, 8), i(4), out=big[:4])
    with pytest.raises(ValueError, match="lora_b"):
        fg.lora_add(C[:4], big[:4], b(1, 8, 16), b(1, 16, 16), i(4))
    with pytest.raises(fg.FP8GemmError, match="UNSUPPORTED"):
        fg.lora_add(C[:4], big[:4], b(1, 136, 16), b(1, 16, 136), i(4))
    with pytest.raises(TypeError, match="tensor"):
        fg.lora_add(C[:4], big[:4], b(1, 8, 16), b(1, 16, 8), [0, 0, 0, 0])
    with pytest.raises(ValueError, match="stream"):
        fg.moe_combine(torch.zeros(4, 16, dtype=torch.bfloat16), i(4, 2), stream=torch.cuda.Stream())


# ------------------------------------------------------------------------------------- together
def layer_inputs(T, E, K, H, N, seed):
    g = gen(seed)
    x = torch.randn(T, K, generator=g).to(torch.bfloat16)
    logits = torch.randn(T, E, generator=g).to(torch.bfloat16)
    w = (torch.randn(E, N, K, generator=g) / K ** 0.5).to(torch.bfloat16)
    return x, logits, w


def layer(fg, x, logits, B, sfb, E, k, masked, stream=None, mmax=None):
    ids, weights, counts, loss, slope = fg.moe_route(logits, k, stream=stream)
    if masked:
        rows, masked_m = fg.moe_layout_masked(ids, E, mmax, stream=stream)
        A, sfa = fg.moe_dispatch_fp8(x, rows, shape=(E, mmax), stream=stream)
        C = fg.m_grouped_gemm_fp8_fp8_bf16_nt_masked(A, sfa, B, sfb, masked_m, stream=stream)
    else:
        rows, m_indices = fg.moe_layout_contiguous(ids, E, stream=stream)
        A, sfa = fg.moe_dispatch_fp8(x, rows, shape=m_indices.numel(), stream=stream)
        C = fg.m_grouped_gemm_fp8_fp8_bf16_nt_contiguous(A, sfa, B, sfb, m_indices, stream=stream)
    return ids, weights, loss, fg.moe_combine(C, rows, weights, stream=stream)


def layer_reference(x, logits, w, k):
    """From the definitions: 64-bit router, the oracle's casts, each product rounded to bf16 once."""
    r = ref.route(f64(logits)[None], k)
    bits = lambda t: t.view(torch.int16).numpy().view(np.uint16)  # noqa: E731
    qx, sx = oracle.quantize_rows(bits(x))
    qw, sw = oracle.quantize_blocks(bits(w))
    T, K = x.shape
    E, N = w.shape[:2]
    table = oracle.e4m3_decode_table()
    dx = table[qx].astype(np.float64) * np.repeat(sx[:, :T].T, 128, 1)[:, :K]
    out, size = np.zeros((T, N)), np.zeros((T, N))
    for e in range(E):
        dw = table[qw[e]].astype(np.float64) * np.repeat(np.repeat(sw[e], 128, 0), 128, 1)[:N, :K]
        y, big = dx @ dw.T, np.abs(dx) @ np.abs(dw).T
        for t in range(T):
            for j in range(k):
                if r["ids"][0, t, j] == e:
                    wt = r["weights"][0, t, j]
                    out[t] += wt * y[t]
                    size[t] += wt * (BF16 * np.abs(y[t]) + 2.0 ** -13 * big[t])  # FP8 sums keep 13 bits or more
    return r, out, size


@pytest.mark.parametrize("masked", [False, True])
def test_a_layer_of_experts(fg, masked):
    T, E, K, N, k = 70, 6, 400, 264, 2
    x, logits, w = layer_inputs(T, E, K, None, N, 11)
    B, sfb = fg.cast_fp8_blocks(w.cuda())
    r, want, size = layer_reference(x, logits, w, k)
    ids, weights, loss, y = layer(fg, x.cuda(), logits.cuda(), B, sfb, E, k, masked, mmax=T)
    assert np.array_equal(ids.cpu().numpy(), r["ids"][0])
    assert np.all(np.abs(f64(y) - want) <= size + BF16 * np.abs(want) + 1e-6 * np.abs(want).max())


def test_adapters_beside_a_projection(fg):
    M, K, N, R, L = 20, 384, 264, 16, 3
    case = lora_case(M, K, N, R, L)
    w = (torch.randn(N, K, generator=gen(1)) / K ** 0.5).to(torch.bfloat16).cuda()
    A, sfa = fg.cast_fp8_rows(case["x"].cuda())
    B, sfb = fg.cast_fp8_blocks(w)
    C = fg.gemm_fp8_fp8_bf16_nt(A, sfa, B, sfb)
    case["C"] = C.cpu()
    dev = {n: t.cuda() for n, t in case.items()}
    # right behind the projection on its stream, in place
    C = fg.gemm_fp8_fp8_bf16_nt(A, sfa, B, sfb)
    fg.lora_add(**{**dev, "C": C}, out=C)
    lora_check(C, case, K, R)


@pytest.mark.parametrize("masked", [False, True])
def test_layer_in_a_graph_replayed_with_new_tokens(fg, masked):
    T, E, K, N, k = 50, 5, 256, 136, 2
    x, logits, w = (t.cuda() for t in layer_inputs(T, E, K, None, N, 12))
    B, sfb = fg.cast_fp8_blocks(w)
    layer(fg, x, logits, B, sfb, E, k, masked, mmax=T)  # first calls outside the capture
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = layer(fg, x, logits, B, sfb, E, k, masked, mmax=T)
    for seed in (13, 14):
        new = layer_inputs(T, E, K, None, N, seed)
        x.copy_(new[0])
        logits.copy_(new[1])
        graph.replay()
        torch.cuda.synchronize()
        want = layer(fg, x, logits, B, sfb, E, k, masked, mmax=T)
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_two_graphs_and_two_streams_at_once(fg):
    """Scratch belongs to the call: two captured graphs and eager calls on two streams do not meet."""
    T, E, k = 3000, 64, 8
    inputs = [torch.randn(T, E, generator=gen(s)).cuda() for s in (1, 2)]
    cases = [{n: t.cuda() for n, t in lora_case(600, 272, 264, 16, 7, s).items()} for s in (1, 2)]

    def step(i, stream=None):
        r = fg.moe_route(inputs[i], k, stream=stream)
        return (*r, *fg.moe_layout_contiguous(r[0], E, stream=stream), fg.lora_add(**cases[i], stream=stream))

    want = [step(i) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    graphs, outs = [], []
    for i in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i], stream=streams[i]):
            outs.append(step(i))
    for _ in range(20):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(a, b) for a, b in zip(outs[i], want[i]))
    for _ in range(10):
        got = [step(i, streams[i]) for i in range(2)]
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(a, b) for a, b in zip(got[i], want[i]))


def test_backward_captured_beside_an_eager_call(fg):
    logits = torch.randn(2, 100, 32, generator=gen(8)).cuda()
    ids, weights, _, loss, slope = fg.moe_route(logits, 4)
    gw, gl = torch.randn_like(weights), torch.ones_like(loss)
    want = fg.moe_route_backward(logits, ids, slope, gw, gl)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = fg.moe_route_backward(logits, ids, slope, gw, gl)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want)


# ------------------------------------------------------------------------------------- long offsets
def test_offsets_past_32_bits(fg):
    """Rows behind 2^31 elements of the expert buffers, and adapters behind 2^31 weights."""
    N, M = 7168, 300_032
    rows = torch.tensor([[0, M - 1], [M - 2, -1]], dtype=torch.int32, device="cuda")
    x = torch.randn(2, N, device="cuda").to(torch.bfloat16)
    q, s = fg.cast_fp8_rows(x)
    A = torch.zeros(M, N, dtype=torch.uint8, device="cuda")
    sfa = torch.zeros(56, M, device="cuda")
    fg.moe_dispatch_fp8(x, rows, A=A, sfa=sfa)
    for t, r in ((0, 0), (0, M - 1), (1, M - 2)):
        assert torch.equal(A[r], q[t]) and torch.equal(sfa[:, r], s[:, t])
    assert not A[1].any() and not A[M - 3].any()
    del A, sfa
    C = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
    C[0], C[M - 1], C[M - 2] = 1.0, 2.0, 4.0
    w = torch.full((2, 2), 0.5, device="cuda")
    out = fg.moe_combine(C, rows, w).float()
    assert (out[0] == 1.5).all() and (out[1] == 2.0).all()
    grad_C = torch.zeros_like(C)
    grad_w = fg.moe_combine_backward(x, C, rows, w, grad_C=grad_C)[1]
    assert torch.equal(grad_C[M - 2], (0.5 * x[1].float()).to(torch.bfloat16)) and not grad_C[M - 3].any()
    assert abs(grad_w[1, 0].item() - 4 * x[1].double().sum().item()) <= (N / 8 + 40) * U * 4 * x[1].double().abs().sum()
    del C, grad_C
    L, R, K, N = 20_000, 16, 7168, 64
    case = lora_case(4, K, N, R, 2)
    case["adapters"] = torch.tensor([1, 0, -1, 1], dtype=torch.int32)
    big = torch.zeros(L, R, K, dtype=torch.bfloat16, device="cuda")
    big[L - 2:] = case["lora_a"].cuda()
    big_b = torch.zeros(L, N, R, dtype=torch.bfloat16, device="cuda")
    big_b[L - 2:] = case["lora_b"].cuda()
    scaling = torch.ones(L, device="cuda")
    scaling[L - 2:] = case["scaling"].cuda()
    ids = torch.where(case["adapters"] >= 0, case["adapters"] + L - 2, -1).to(torch.int32).cuda()
    got = fg.lora_add(case["C"].cuda(), case["x"].cuda(), big, big_b, ids, scaling)
    lora_check(got, case, K, R)

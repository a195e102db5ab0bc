"""The operators around the grouped GEMMs as cases to measure: plain forms, the library's calls, and values in 64 bits.

  route     top-k choice of experts with its weights, per-expert counts and the balance loss
            (train: with the gradient of the logits)
  dispatch  the rows of the experts' layout (contiguous or masked) and the rows cast to FP8 into it
  combine   the weighted sum of the experts' output rows of each token (train: with its gradients)
  lora      low-rank adapters of many requests beside a shared projection

own = False computes the plain forms in elementary torch operations; own = True calls the package.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
ALIGN = 128  # rows that an expert's block of the contiguous layout is padded to


def cdiv(a, b):
    return (a + b - 1) // b


def layout_rows(pairs, experts):
    """Rows of a contiguous layout that hold any choice of `pairs` rows among `experts`."""
    n = min(pairs, experts)
    return ALIGN * (n + (pairs - n) // ALIGN)


def scale_ld(rows):
    return cdiv(rows, 4) * 4


# ------------------------------------------------------------------------------------- the cases
def listed():
    return [
        # the router of one decode step: a batch of single tokens, fp32 logits
        dict(name="route_decode", op="route", train=False, seqs=1, tokens=64, experts=256, k=8, dtype="fp32",
             renorm=True, masked=0.0, closed=0.0),
        # odd sizes, some experts closed to some tokens, weights not renormalised
        dict(name="route_odd", op="route", train=True, seqs=3, tokens=1537, experts=60, k=4, dtype="fp16",
             renorm=False, masked=0.1, closed=0.3),
        # a training batch: padded sequences, each with its own balance loss, forward and backward
        dict(name="route_train", op="route", train=True, seqs=8, tokens=4096, experts=256, k=8, dtype="bf16",
             renorm=True, masked=0.1, closed=0.0),
        # one decode step on a rank that holds 32 of 256 experts, masked layout
        dict(name="dispatch_decode", op="dispatch", masked=True, tokens=64, k=8, experts=32, total=256, mmax=64,
             K=7168, fmt="e4m3"),
        # ragged: odd token and expert counts, a partial last K block, the other format
        dict(name="dispatch_odd", op="dispatch", masked=False, tokens=777, k=3, experts=5, total=5, mmax=0, K=2064,
             fmt="e5m2"),
        # the rows of the contiguous benchmark shape with 8 experts (about 4096 rows each)
        dict(name="dispatch_prefill", op="dispatch", masked=False, tokens=16384, k=2, experts=8, total=8, mmax=0,
             K=7168, fmt="e4m3"),
        # back from the masked layout, one decode step
        dict(name="combine_decode", op="combine", train=False, masked=True, tokens=64, k=8, experts=32, total=256,
             mmax=64, N=7168),
        # back from the contiguous layout, prefill
        dict(name="combine_prefill", op="combine", train=False, masked=False, tokens=16384, k=2, experts=8, total=8,
             mmax=0, N=7168),
        # a training step's sum and its gradients
        dict(name="combine_train", op="combine", train=True, masked=False, tokens=4096, k=8, experts=64, total=64,
             mmax=0, N=2048),
        # a single request's token
        dict(name="lora_token", op="lora", rows=1, K=7168, N=4096, R=16, adapters=4, runs=False, bare=0.0),
        # a decode batch, every request with an adapter of its own choice, a few without
        dict(name="lora_decode", op="lora", rows=128, K=7168, N=4096, R=16, adapters=64, runs=False, bare=0.1),
        # prompts of several requests one after the other
        dict(name="lora_prefill", op="lora", rows=4096, K=7168, N=4096, R=64, adapters=8, runs=True, bare=0.1),
    ]


def spread(rng, low, high):
    """A whole number spread over the logarithm of [low, high]."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["route", "dispatch", "combine", "lora"])
    if op == "route":
        experts = spread(rng, 2, 512)
        seqs = rng.randint(1, 8)
        return dict(op=op, train=rng.random() < 0.5, seqs=seqs, tokens=spread(rng, 1, min(4096, 8388608 // (experts * seqs))),
                    experts=experts, k=rng.randint(1, min(experts, 10)), dtype=rng.choice(["fp32", "bf16", "fp16"]),
                    renorm=rng.random() < 0.5, masked=rng.choice([0.0, 0.1, 0.6]), closed=rng.choice([0.0, 0.3]))
    if op in ("dispatch", "combine"):
        masked = rng.random() < 0.4
        k = rng.randint(1, 8)
        experts = spread(rng, 1, 32 if masked else 128)
        total = experts * rng.choice([1, 1, 4])
        k = min(k, total)
        tokens = spread(rng, 1, 256) if masked else spread(rng, 1, 16384 // k)
        width = 16 * spread(rng, 8, 448)
        case = dict(op=op, masked=masked, tokens=tokens, k=k, experts=experts, total=total,
                    mmax=spread(rng, max(1, tokens // 2), tokens) if masked else 0)
        if op == "dispatch":
            case.update(K=width, fmt=rng.choice(["e4m3", "e4m3", "e5m2"]))
        else:
            case.update(N=width, train=rng.random() < 0.5)
        return case
    rank = 8 * rng.randint(1, 12)
    rows = spread(rng, 1, 4096)
    return dict(op=op, rows=rows, K=16 * spread(rng, 8, 448), N=16 * spread(rng, 8, 448), R=rank,
                adapters=spread(rng, 1, max(1, min(64, 2097152 // (rows * rank)))), runs=rng.random() < 0.5,
                bare=rng.choice([0.0, 0.1, 0.5]))


# ------------------------------------------------------------------------------------- the inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return {"route": prepare_route, "dispatch": prepare_dispatch, "combine": prepare_combine,
            "lora": prepare_lora}[case["op"]](case, g)


def normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def uniform(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda")


def prepare_route(case, g):
    S, T, E, k = case["seqs"], case["tokens"], case["experts"], case["k"]
    logits = 1.5 * normal(g, S, T, E) + 0.5 * normal(g, E)
    if case["closed"]:
        logits = logits.masked_fill(uniform(g, S, T, E) < case["closed"], -math.inf)
    logits = logits.to(DTYPES[case["dtype"]])
    mask = None
    if case["masked"]:  # padding behind each sequence's end; whatever stands there is not read as a logit
        ends = (T * (1 - 2 * case["masked"] * uniform(g, S, 1))).clamp(min=0)
        mask = torch.arange(T, device="cuda") < ends
        junk = torch.tensor([math.nan, math.inf, torch.finfo(logits.dtype).min, -math.inf], device="cuda")
        junk = junk.to(logits.dtype)[torch.arange(E, device="cuda") % 4]
        logits = torch.where(mask[..., None], logits, junk)
    return dict(case=case, logits=logits, mask=mask, grad_weights=normal(g, S, T, k),
                grad_loss=0.01 * T * (1 + uniform(g, S)))


def choose(case, g):
    """Expert choices [tokens, k] of a skewed router; those of other ranks are -1."""
    T, k, E, total = case["tokens"], case["k"], case["experts"], case["total"]
    liked = normal(g, T, total) + 0.7 * normal(g, total)
    ids = liked.topk(k, dim=1).indices.to(torch.int32)
    return torch.where(ids < E, ids, -1)


def prepare_dispatch(case, g):
    T, K, E = case["tokens"], case["K"], case["experts"]
    x = (normal(g, T, K) * torch.exp(2 * normal(g, T, 1))).to(torch.bfloat16)
    KB = cdiv(K, 128)
    if case["masked"]:
        shape, scales = (E, case["mmax"], K), (E, KB, scale_ld(case["mmax"]))
    else:
        M = layout_rows(T * case["k"], E)
        shape, scales = (M, K), (KB, scale_ld(M))
    # the layout's buffers, kept over the calls: rows that no token takes stay as they are
    return dict(case=case, x=x, ids=choose(case, g), A=torch.zeros(shape, dtype=torch.uint8, device="cuda"),
                sfa=torch.zeros(scales, device="cuda"))


def prepare_combine(case, g):
    T, N, E = case["tokens"], case["N"], case["experts"]
    ids = choose(case, g)
    rows = layout_plain(case, ids)[0]
    shape = (E, case["mmax"], N) if case["masked"] else (layout_rows(T * case["k"], E), N)
    weights = uniform(g, T, case["k"]) + 0.05
    state = dict(case=case, C=normal(g, *shape).to(torch.bfloat16), rows=rows,
                 weights=weights / weights.sum(1, keepdim=True))
    if case["train"]:
        state.update(grad_out=normal(g, T, N).to(torch.bfloat16),
                     grad_C=torch.zeros(shape, dtype=torch.bfloat16, device="cuda"))
    return state


def prepare_lora(case, g):
    M, K, N, R, L = case["rows"], case["K"], case["N"], case["R"], case["adapters"]
    if case["runs"]:  # requests one after the other, each a run of rows
        cuts = torch.sort(uniform(g, max(L - 1, 0))).values * M
        which = torch.randperm(L, generator=g, device="cuda")
        ids = which[(torch.arange(M, device="cuda")[:, None] >= cuts).sum(1)]
        ids = torch.where(uniform(g, L)[ids] < case["bare"], -1, ids)
    else:
        ids = torch.randint(0, L, (M,), generator=g, device="cuda")
        ids = torch.where(uniform(g, M) < case["bare"], -1, ids)
    return dict(case=case, C=normal(g, M, N).to(torch.bfloat16), x=normal(g, M, K).to(torch.bfloat16),
                lora_a=(normal(g, L, R, K) / math.sqrt(K)).to(torch.bfloat16),
                lora_b=(normal(g, L, N, R) / math.sqrt(R)).to(torch.bfloat16), ids=ids.to(torch.int32),
                scaling=0.5 + uniform(g, L), out=torch.empty(M, N, dtype=torch.bfloat16, device="cuda"))


# ------------------------------------------------------------------------------------- one pass
def run(state):
    op = state["case"]["op"]
    if own:
        return {"route": route_own, "dispatch": dispatch_own, "combine": combine_own, "lora": lora_own}[op](state)
    return {"route": route_plain, "dispatch": dispatch_plain, "combine": combine_plain, "lora": lora_plain}[op](state)


def route_own(s):
    import moe_grouped_gemm_08_b200 as fg
    c = s["case"]
    ids, weights, counts, loss, slope = fg.moe_route(s["logits"], c["k"], mask=s["mask"], renormalize=c["renorm"])
    out = dict(ids=ids, weights=weights, counts=counts, loss=loss)
    if c["train"]:
        out["grad"] = fg.moe_route_backward(s["logits"], ids, slope, s["grad_weights"], s["grad_loss"],
                                            renormalize=c["renorm"])
    return out


def dispatch_own(s):
    import moe_grouped_gemm_08_b200 as fg
    c = s["case"]
    if c["masked"]:
        rows, group = fg.moe_layout_masked(s["ids"], c["experts"], c["mmax"])
    else:
        rows, group = fg.moe_layout_contiguous(s["ids"], c["experts"])
    A, sfa = fg.moe_dispatch_fp8(s["x"], rows, A=s["A"], sfa=s["sfa"], fmt=c["fmt"])
    return dict(rows=rows, group=group, A=A.view(float8(c["fmt"])), sfa=sfa)


def combine_own(s):
    import moe_grouped_gemm_08_b200 as fg
    out = [fg.moe_combine(s["C"], s["rows"], s["weights"])]
    if s["case"]["train"]:
        out += fg.moe_combine_backward(s["grad_out"], s["C"], s["rows"], s["weights"], grad_C=s["grad_C"])
    return out


def lora_own(s):
    import moe_grouped_gemm_08_b200 as fg
    return fg.lora_add(s["C"], s["x"], s["lora_a"], s["lora_b"], s["ids"], scaling=s["scaling"], out=s["out"])


# ------------------------------------------------------------------------------------- plain forms
def route_plain(s):
    c, E, k = s["case"], s["case"]["experts"], s["case"]["k"]
    l = s["logits"].float()
    if s["mask"] is not None:
        l = l.masked_fill(~s["mask"][..., None], -math.inf)
    order = torch.sort(l, dim=-1, descending=True, stable=True)
    top = order.values[..., :k]
    chosen = top > -math.inf
    ids = torch.where(chosen, order.indices[..., :k], -1).to(torch.int32)
    routed = chosen[..., :1]
    high = torch.where(routed, top[..., :1], 0.0)
    e = torch.exp(l - high)
    p = torch.where(routed, e / e.sum(-1, keepdim=True), 0.0)
    at = order.indices[..., :k]
    weights = p.gather(-1, at) * chosen
    if c["renorm"]:
        et = torch.exp(top - high)
        weights = torch.where(chosen, et / et.sum(-1, keepdim=True), 0.0)
    counts = torch.zeros(c["seqs"], E, dtype=torch.int32, device=l.device)
    counts.scatter_add_(1, at.flatten(1), chosen.flatten(1).to(torch.int32))
    tokens = routed.sum((1, 2)).clamp(min=1)
    slope = E * counts / (counts.sum(1).clamp(min=1) * tokens)[:, None]
    out = dict(ids=ids, weights=weights, counts=counts, loss=(slope * p.sum(1)).sum(1))
    if c["train"]:
        h = (s["grad_loss"][:, None] * slope)[:, None, :].expand_as(p)
        gw = s["grad_weights"] * chosen
        if not c["renorm"]:
            h = h.scatter_add(-1, at, gw)
        grad = p * (h - (p * h).sum(-1, keepdim=True))
        if c["renorm"]:
            grad = grad.scatter_add(-1, at, weights * (gw - (weights * gw).sum(-1, keepdim=True)))
        out["grad"] = grad.to(s["logits"].dtype)
    return out


def layout_plain(c, ids):
    """(rows, m_indices) of the contiguous layout, (rows, masked_m) of the masked one."""
    E, flat = c["experts"], ids.flatten().long()
    live = flat >= 0
    key = torch.where(live, flat, E)
    order = torch.sort(key, stable=True).indices
    counts = torch.zeros(E + 1, dtype=torch.int64, device=ids.device).scatter_add_(0, key, torch.ones_like(key))
    place = torch.empty_like(key)
    place[order] = torch.arange(key.numel(), device=ids.device)
    place -= (counts.cumsum(0) - counts)[key]  # the pair's place among those of its expert
    if c["masked"]:
        live &= place < c["mmax"]
        rows = key * c["mmax"] + place
        group = counts[:E].clamp(max=c["mmax"])
    else:
        padded = (counts[:E] + ALIGN - 1) // ALIGN * ALIGN
        start = padded.cumsum(0) - padded
        rows = start[key.clamp(max=E - 1)] + place
        at = torch.arange(layout_rows(key.numel(), E), device=ids.device)
        e = torch.searchsorted(padded.cumsum(0), at, right=True).clamp(max=E - 1)
        group = torch.where(at - start[e] < counts[e], e, -1)
    return torch.where(live, rows, -1).view(ids.shape).to(torch.int32), group.to(torch.int32)


def float8(fmt):
    return torch.float8_e4m3fn if fmt == "e4m3" else torch.float8_e5m2


def dispatch_plain(s):
    c, x = s["case"], s["x"]
    T, K, k = c["tokens"], c["K"], c["k"]
    KB = cdiv(K, 128)
    rows, group = layout_plain(c, s["ids"])
    xf = torch.nn.functional.pad(x.float(), (0, KB * 128 - K)).view(T, KB, 128)
    amax = xf.abs().amax(-1)
    scale = torch.where(amax > 0, amax / (448.0 if c["fmt"] == "e4m3" else 57344.0), 1.0)
    codes = (xf / scale[..., None]).view(T, -1)[:, :K].to(float8(c["fmt"])).view(torch.uint8)
    flat = rows.flatten().long()
    pair = torch.nonzero(flat >= 0).flatten()
    row, token = flat[pair], pair // k
    s["A"].view(-1, K)[row] = codes[token]
    if c["masked"]:
        s["sfa"][row // c["mmax"], :, row % c["mmax"]] = scale[token]
    else:
        s["sfa"][:, row] = scale[token].t()
    return dict(rows=rows, group=group, A=s["A"].view(float8(c["fmt"])), sfa=s["sfa"])


def combine_plain(s):
    c, N = s["case"], s["case"]["N"]
    C = s["C"].view(-1, N)
    live = s["rows"] >= 0
    at = s["rows"].clamp(min=0).long()
    w = s["weights"] * live
    picked = C[at].float() * live[..., None]
    out = [(w[..., None] * picked).sum(1).to(torch.bfloat16)]
    if c["train"]:
        go = s["grad_out"].float()
        pair = torch.nonzero(live.flatten()).flatten()
        s["grad_C"].view(-1, N)[at.flatten()[pair]] = (w[..., None] * go[:, None]).to(torch.bfloat16).flatten(0, 1)[pair]
        out += [s["grad_C"], (picked * go[:, None]).sum(-1)]
    return out


def lora_plain(s):
    c = s["case"]
    L, R = c["adapters"], c["R"]
    h = s["x"].float() @ s["lora_a"].float().view(L * R, -1).t()
    mine = s["ids"][:, None] == torch.arange(L, device=h.device)
    h = h.view(-1, L, R) * (mine * s["scaling"])[..., None]
    delta = h.view(-1, L * R) @ s["lora_b"].float().transpose(1, 2).reshape(L * R, -1)
    torch.add(s["C"].float(), delta, out=delta)
    return s["out"].copy_(delta)


# ------------------------------------------------------------------------------------- work
def work(case):
    if case["op"] == "route":
        n = case["seqs"] * case["tokens"]
        size = 4 if case["dtype"] == "fp32" else 2
        row = n * case["experts"] * size
        out = 8 * n * case["k"]
        total = row + out + 4 * case["seqs"] * case["experts"] + (n if case["masked"] else 0)
        if case["train"]:  # logits again, choices and gradients of the weights in, gradient out
            total += 2 * row + out
        return {"bytes": total, "flops": 5 * n * case["experts"] * (2 if case["train"] else 1)}
    if case["op"] in ("dispatch", "combine"):
        T, k = case["tokens"], case["k"]
        pairs = T * k * case["experts"] / case["total"]
        if case["op"] == "dispatch":
            K = case["K"]
            group = case["experts"] if case["masked"] else layout_rows(T * k, case["experts"])
            return {"bytes": 2 * T * K + 8 * T * k + 4 * group + pairs * (K + 4 * cdiv(K, 128)), "flops": 2 * T * K}
        N = case["N"]
        total = 2 * pairs * N + 2 * T * N + 8 * T * k
        if case["train"]:
            total += 4 * pairs * N + 2 * T * N + 12 * T * k
        return {"bytes": total, "flops": pairs * N * (5 if case["train"] else 2)}
    M, K, N, R, L = case["rows"], case["K"], case["N"], case["R"], case["adapters"]
    live = M * (1 - case["bare"])
    used = min(L, live) if case["runs"] else L * (1 - (1 - 1 / L) ** live) if L > 1 else min(1, live)
    return {"bytes": 2 * live * K + 2 * used * R * (K + N) + 4 * M * N, "flops": 2 * live * R * (K + N)}


# ------------------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    """run()'s outputs from the definitions in float64; None in the place of whole numbers."""
    s = prepare(case, seed)
    return {"route": route_exact, "dispatch": dispatch_exact, "combine": combine_exact,
            "lora": lora_exact}[case["op"]](s)


def route_exact(s):
    c = s["case"]
    S, T, E, k = c["seqs"], c["tokens"], c["experts"], c["k"]
    logits = s["logits"].double().cpu().numpy()
    mask = np.ones((S, T), bool) if s["mask"] is None else s["mask"].cpu().numpy()
    gw, gl = s["grad_weights"].double().cpu().numpy(), s["grad_loss"].double().cpu().numpy()
    weights, loss, grad = np.zeros((S, T, k)), np.zeros(S), np.zeros((S, T, E))
    for q in range(S):
        rows = np.flatnonzero(mask[q] & (np.where(mask[q][:, None], logits[q], -np.inf).max(1) > -np.inf))
        if not rows.size:
            continue
        l = logits[q][rows]
        ids = np.argsort(-l, axis=1, kind="stable")[:, :k]
        open_ = np.isfinite(np.take_along_axis(l, ids, 1))
        e = np.exp(l - l.max(1, keepdims=True))
        p = e / e.sum(1, keepdims=True)
        picked = np.take_along_axis(p, ids, 1) * open_
        w = picked / picked.sum(1, keepdims=True) if c["renorm"] else picked
        weights[q][rows] = w
        hot = np.zeros((rows.size, E))
        np.put_along_axis(hot, ids, open_.astype(float), 1)
        f = hot.sum(0) / hot.sum()
        loss[q] = E * (f * p.mean(0)).sum()
        dp = np.tile(gl[q] * E * f / rows.size, (rows.size, 1))
        dw = gw[q][rows] * open_
        if c["renorm"]:  # w = picked / sum(picked)
            total = picked.sum(1, keepdims=True)
            dw = (dw - (dw * w).sum(1, keepdims=True)) / total * open_
        np.put_along_axis(dp, ids, np.take_along_axis(dp, ids, 1) + dw, 1)
        grad[q][rows] = p * (dp - (p * dp).sum(1, keepdims=True))
    out = dict(ids=None, weights=weights, counts=None, loss=loss)
    if c["train"]:
        out["grad"] = grad
    return out


def round8(v, fmt):
    """Nearest FP8 value of each float64 (ties to even), saturating."""
    bits, least, top = (3, -6, 448.0) if fmt == "e4m3" else (2, -14, 57344.0)
    exponent = (torch.frexp(v).exponent - 1).clamp(min=least)
    step = torch.ldexp(torch.ones_like(v), exponent - bits)
    return (torch.round(v / step) * step).clamp(-top, top)


def dispatch_exact(s):
    c = s["case"]
    K, k = c["K"], c["k"]
    KB = cdiv(K, 128)
    rows = layout_plain(c, s["ids"])[0].flatten().long()
    A = s["A"].view(-1, K).to(torch.float32)
    sfa = s["sfa"].double()
    top = 448.0 if c["fmt"] == "e4m3" else 57344.0
    pair = torch.nonzero(rows >= 0).flatten()
    row, x = rows[pair], s["x"].double()[pair // k]
    for b in range(KB):
        block = x[:, 128 * b:128 * (b + 1)]
        scale = block.abs().amax(1) / top
        scale[scale == 0] = 1.0
        A[row, 128 * b:128 * (b + 1)] = round8(block / scale[:, None], c["fmt"]).float()
        if c["masked"]:
            sfa[row // c["mmax"], b, row % c["mmax"]] = scale
        else:
            sfa[b, row] = scale
    return dict(rows=None, group=None, A=A.view(s["A"].shape), sfa=sfa)


def combine_exact(s):
    c, N = s["case"], s["case"]["N"]
    C, rows, w = s["C"].view(-1, N), s["rows"].long(), s["weights"].double()
    out = torch.zeros(c["tokens"], N, dtype=torch.float64, device=w.device)
    grad_w = torch.zeros_like(w)
    for j in range(c["k"]):
        t = torch.nonzero(rows[:, j] >= 0).flatten()
        row = C[rows[t, j]].double()
        out[t] += w[t, j][:, None] * row
        if c["train"]:
            grad_w[t, j] = (row * s["grad_out"][t].double()).sum(1)
    if not c["train"]:
        return [out]
    grad_C = torch.zeros(C.shape, dtype=torch.float64, device=w.device)
    for j in range(c["k"]):
        t = torch.nonzero(rows[:, j] >= 0).flatten()
        grad_C[rows[t, j]] = w[t, j][:, None] * s["grad_out"][t].double()
    return [out, grad_C.view(s["C"].shape), grad_w]


def lora_exact(s):
    out = s["C"].double()
    for a in range(s["case"]["adapters"]):
        m = torch.nonzero(s["ids"] == a).flatten()
        h = s["x"][m].double() @ s["lora_a"][a].double().t() * s["scaling"][a].double()
        out[m] += h @ s["lora_b"][a].double().t()
    return out

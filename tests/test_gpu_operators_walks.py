"""GPU tests of the operators around the GEMMs at sizes where every loop of a kernel takes three steps or more: rings
of shared memory that wrap, both buffers of TMEM and their barriers' phases, rows loaded ahead, state of a
row that has to be cleared for the next, CTAs that walk over several tokens.  Plain forms in float64 on the
device, from the definitions in include/fp8gemm.h; sizes are stated for 148 SMs.

Tolerances: u = 2^-24 for each fp32 rounding behind a value, half a step of the output's type for the
last one; products on the tensor cores are exact and each of their accumulations loses up to 2 u of the
sum of sizes.
"""
from __future__ import annotations

import pytest
import torch

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


@pytest.fixture(autouse=True)
def _give_back_memory():
    yield
    torch.cuda.empty_cache()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def holds(err, tol):
    over = err - tol
    assert bool((over <= 0).all()), (over.max().item(), int((over > 0).sum()))


# ------------------------------------------------------------------------------------- adapters
def adapters_case(M, K, N, R, L, seed):
    g = gen(seed)
    return dict(C=normal(g, M, N).to(torch.bfloat16), x=normal(g, M, K).to(torch.bfloat16),
                lora_a=(normal(g, L, R, K) / K ** 0.5).to(torch.bfloat16), lora_b=normal(g, L, N, R).to(torch.bfloat16),
                adapters=torch.randint(-1, L, (M,), generator=g, device="cuda").to(torch.int32), scaling=normal(g, L))


def adapters_want(c):
    """(out, tolerance): h carries K / 16 + 40 accumulations, the second product three parts of R / 16 steps."""
    R, K = c["lora_a"].shape[1:]
    out, tol = c["C"].double(), torch.zeros(c["C"].shape, dtype=torch.float64, device="cuda")
    for i in range(c["lora_a"].shape[0]):
        m = torch.nonzero(c["adapters"] == i).flatten()
        s, a, b, x = c["scaling"][i].double(), c["lora_a"][i].double(), c["lora_b"][i].double(), c["x"][m].double()
        h = x @ a.t() * s
        out[m] += h @ b.t()
        tol[m] = (2 * (K / 16 + 40) * U * (x.abs() @ a.t().abs() * s.abs()) + 2 * (3 * R / 16 + 8) * U * h.abs()) @ b.t().abs()
    return out, tol * (1 + BF16) + BF16 * out.abs()


@pytest.mark.parametrize("M,K,N,R,L", [
    # by rank, over the adapters' tiles: lora_down_kernel 13 or 27 units a CTA (its ring holds 4 to 6),
    # lora_up_kernel 7 or 15 chunks (its ring holds 3 or 4)
    (4000, 7168, 4096, 16, 4), (4000, 7168, 4096, 32, 5), (4000, 7168, 4096, 64, 3), (4000, 7168, 4096, 128, 6),
    # one tile's h from many CTAs; many tiles a CTA, with parts of tiles at both ends
    (300, 16384, 9992, 24, 1), (20000, 400, 712, 40, 2), (9000, 1040, 1000, 72, 700), (30000, 144, 2056, 8, 30),
])
def test_adapters_of_many_rows(fg, M, K, N, R, L):
    case = adapters_case(M, K, N, R, L, M + R)
    want, tol = adapters_want(case)
    out = fg.lora_add(**case)
    holds((out.double() - want).abs(), tol)
    none = case["adapters"] < 0
    assert torch.equal(out[none], case["C"][none])
    assert torch.equal(fg.lora_add(**case, out=case["C"]), out)
    assert fg.lora_status() == 0


@pytest.mark.parametrize("M,K,N,R,L", [(3, 40016, 40008, 16, 1), (64, 20000, 9992, 128, 3), (200, 20000, 9992, 40, 7),
                                       (150, 24000, 16392, 8, 2), (90, 30000, 16392, 32, 90)])
def test_adapters_of_few_rows(fg, M, K, N, R, L):
    """Each warp takes several steps over K and over N."""
    case = adapters_case(M, K, N, R, L, M + R)
    want, tol = adapters_want(case)
    out = fg.lora_add(**case)
    holds((out.double() - want).abs(), tol)
    assert torch.equal(fg.lora_add(**case, out=case["C"]), out)


@pytest.mark.parametrize("M", [64, 700, 3000])
@pytest.mark.parametrize("R", [16, 128])
def test_adapters_right_behind_a_projection(fg, M, R):
    """In place on the GEMM's output, launched before the GEMM has run: the same bits as with a wait between, for
    inputs that change from pass to pass."""
    K, N, L = 1040, 1032, 6
    case = adapters_case(M, K, N, R, L, M + R)
    B, sfb = fg.cast_fp8_blocks((normal(gen(1), N, K) / K ** 0.5).to(torch.bfloat16))
    inputs = [case["x"] * s for s in (1.0, -0.5, 2.0, 0.25)]
    cast = [fg.cast_fp8_rows(x) for x in inputs]
    ids = [case["adapters"].roll(i) for i in range(4)]
    want = []
    for x, (A, sfa), a in zip(inputs, cast, ids):
        C = fg.gemm_fp8_fp8_bf16_nt(A, sfa, B, sfb)
        torch.cuda.synchronize()
        want.append(fg.lora_add(**{**case, "C": C, "x": x, "adapters": a}))
        torch.cuda.synchronize()
    for _ in range(5):
        got = []
        C = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
        for x, (A, sfa), a in zip(inputs, cast, ids):
            fg.gemm_fp8_fp8_bf16_nt(A, sfa, B, sfb, C=C)
            fg.lora_add(**{**case, "C": C, "x": x, "adapters": a}, out=C)
            got.append(C.clone())
            a.add_(0)  # a kernel of torch between
        for one, other in zip(got, want):
            assert torch.equal(one, other)


# ------------------------------------------------------------------------------------- the router
def route_want(logits, k, mask, renorm):
    l = logits.double()
    if mask is not None:
        l = l.masked_fill(~mask[..., None], -torch.inf)
    top, at = torch.sort(l, dim=-1, descending=True, stable=True)
    top, at = top[..., :k], at[..., :k]
    chosen = top > -torch.inf
    routed = chosen[..., :1]
    e = torch.exp(l - torch.where(routed, top[..., :1], 0.0))
    p = torch.where(routed, e / e.sum(-1, keepdim=True), 0.0)
    picked = p.gather(-1, at) * chosen
    weights = torch.where(chosen, picked / picked.sum(-1, keepdim=True), 0.0) if renorm else picked
    S, _, E = l.shape
    counts = torch.zeros(S, E, dtype=torch.int64, device="cuda").scatter_add_(1, at.flatten(1), chosen.flatten(1).long())
    slope = E * counts.double() / (counts.sum(1) * routed.sum((1, 2))).clamp(min=1)[:, None]
    return dict(ids=torch.where(chosen, at, -1).int(), at=at, chosen=chosen, weights=weights, counts=counts.int(),
                slope=slope, loss=(slope * p.sum(1)).sum(1), p=p)


def route_gradient_want(w, gw, gl, renorm):
    """(gradient, sums of the sizes behind it)"""
    p, at, g = w["p"], w["at"], gw.double() * w["chosen"]
    h = (gl.double()[:, None] * w["slope"])[:, None].expand_as(p)
    if not renorm:
        h = h.scatter_add(-1, at, g)
    grad = p * (h - (p * h).sum(-1, keepdim=True))
    size = p * (h.abs() + (p * h.abs()).sum(-1, keepdim=True))
    if renorm:
        v = w["weights"]
        grad = grad.scatter_add(-1, at, v * (g - (v * g).sum(-1, keepdim=True)))
        size = size.scatter_add(-1, at, v * (g.abs() + (v * g.abs()).sum(-1, keepdim=True)))
    return grad, size


ROUTES = [  # S, T, E, k, dtype, renorm, misaligned base.  Rows a CTA takes at once: 32 up to 64 experts, 16 up to 128, else 8
    (1, 100_001, 5, 2, "fp32", True, False), (3, 40_003, 32, 4, "fp16", False, False), (1, 120_001, 64, 6, "bf16", True, False),
    (2, 60_001, 60, 9, "fp16", True, False), (1, 100_001, 64, 8, "fp32", False, False), (2, 60_001, 64, 7, "bf16", True, True),
    (2, 20_001, 96, 6, "fp32", True, False), (1, 61_001, 128, 8, "bf16", False, False), (3, 15_001, 120, 8, "fp32", True, True),
    (1, 20_001, 256, 8, "fp32", True, False), (8, 4_001, 256, 8, "bf16", True, False), (1, 30_001, 250, 3, "fp16", False, False),
    (2, 15_001, 256, 12, "fp16", True, True), (1, 20_001, 512, 16, "bf16", True, False), (1, 20_001, 400, 5, "fp32", False, True),
    (1, 20_001, 1000, 32, "fp32", True, False), (2, 10_001, 1024, 8, "bf16", True, False), (1, 20_001, 777, 4, "fp16", True, False),
]


@pytest.mark.parametrize("S,T,E,k,dtype,renorm,misaligned", ROUTES)
def test_router_of_many_tokens(fg, S, T, E, k, dtype, renorm, misaligned):
    g = gen(T + E)
    values = 1.5 * normal(g, S, T, E)
    values = values.masked_fill(torch.rand(S, T, E, generator=g, device="cuda") < 0.1, -torch.inf)
    values[:, T // 3] = -torch.inf
    buffer = torch.zeros(S * T * E + 1, dtype=DTYPES[dtype], device="cuda")
    logits = buffer[1:].view(S, T, E) if misaligned else buffer[:-1].view(S, T, E)
    logits.copy_(values)
    del values
    mask = torch.rand(S, T, generator=g, device="cuda") < 0.8
    mask[:, T // 2:T // 2 + 200] = False  # whole warps and CTAs without a token
    logits[~mask] = torch.tensor([torch.nan, torch.inf, -torch.inf, 3.0], device="cuda").to(logits.dtype).repeat(E)[:E]
    want = route_want(logits, k, mask, renorm)
    ids, weights, counts, loss, slope = fg.moe_route(logits, k, mask=mask, renormalize=renorm)
    assert torch.equal(ids, want["ids"]) and torch.equal(counts, want["counts"])
    # a softmax term: the difference rounds an argument of at most 20, e^x 2 ulp, its sum 40 additions, a division
    rel = (20 + 4 + 40 + 2) * U
    holds((weights.double() - want["weights"]).abs(), 2 * rel * want["weights"])
    holds((slope.double() - want["slope"]).abs(), 4 * U * want["slope"])
    # the loss: sums over rows of a lane (at most T / 148 / 4), lanes, chunks (eight per SM) and experts
    holds((loss.double() - want["loss"]).abs(), (rel + (T / 592 + 40 + 1200 + E) * U) * want["loss"])
    gw, gl = normal(g, S, T, k), 1000 * normal(g, S)
    half, least = torch.finfo(logits.dtype).eps / 2, torch.finfo(logits.dtype).smallest_normal
    for use_w, use_l in ((True, True), (True, False), (False, True)):
        got = fg.moe_route_backward(logits, ids, slope, gw if use_w else None, gl if use_l else None, renormalize=renorm)
        grad, size = route_gradient_want(want, gw * use_w, gl * use_l, renorm)
        holds((got.double() - grad).abs(), (4 * rel + 80 * U) * size * (1 + half) + half * grad.abs() + 2 * half * least)
        assert not bool(got[want["ids"][..., 0] < 0].any())


# ------------------------------------------------------------------------------------- rows
def layout_case(fg, T, k, E, seed, none=0.1):
    g = gen(seed)
    ids = torch.rand(T, E, generator=g, device="cuda").topk(k, dim=1).indices.int()
    ids = torch.where(torch.rand(T, k, generator=g, device="cuda") < none, -1, ids)
    ids[T // 3:T // 3 + 40] = -1
    return g, *fg.moe_layout_contiguous(ids, E)


@pytest.mark.parametrize("T,k,E,K,fmt", [(200_001, 2, 5, 16, "e4m3"), (60_000, 4, 16, 2064, "e5m2"), (150_003, 9, 9, 272, "e4m3")])
def test_dispatch_of_many_tokens(fg, T, k, E, K, fmt):
    """A warp takes three tokens or more (47360 warps at once)."""
    g, rows, group = layout_case(fg, T, k, E, T)
    x = (normal(g, T, K) * torch.exp(2 * normal(g, T, 1))).to(torch.bfloat16)
    M = group.numel()
    A = torch.full((M, K), 0xA5, dtype=torch.uint8, device="cuda")
    sfa = torch.full((-(-K // 128), fg.sfa_ld(M)), -7.0, device="cuda")
    fg.moe_dispatch_fp8(x, rows, A=A, sfa=sfa, fmt=fmt)
    q, s = fg.cast_fp8_rows(x, fmt=fmt)
    want_A, want_s = torch.full_like(A, 0xA5), torch.full_like(sfa, -7.0)
    for j in range(k):
        t = torch.nonzero(rows[:, j] >= 0).flatten()
        want_A[rows[t, j].long()] = q[t]
        want_s[:, rows[t, j].long()] = s[:, t]
    assert torch.equal(A, want_A) and torch.equal(sfa, want_s)


@pytest.mark.parametrize("T,k,E,N", [(12_001, 1, 4, 264), (12_001, 2, 8, 4104), (12_001, 4, 16, 1032), (12_001, 8, 8, 264),
                                     (6_001, 8, 64, 4104), (12_001, 9, 9, 1040), (3_001, 17, 20, 4104), (40_001, 3, 3, 16)])
def test_combine_of_many_tokens(fg, T, k, E, N):
    """Each warp and CTA takes three tokens or more (3552 and 444 at once); N passes one span of the gradient's CTA."""
    g, rows, group = layout_case(fg, T, k, E, T + k)
    M = group.numel()
    C = normal(g, M, N).to(torch.bfloat16)
    C[group < 0] = torch.nan  # rows of no choice are not read
    weights, go = normal(g, T, k), normal(g, T, N).to(torch.bfloat16)
    out, size = (torch.zeros(T, N, dtype=torch.float64, device="cuda") for _ in range(2))
    grad_C = torch.full((M, N), 3.0, dtype=torch.float64, device="cuda")
    grad_w, size_w = (torch.zeros(T, k, dtype=torch.float64, device="cuda") for _ in range(2))
    for j in range(k):
        t = torch.nonzero(rows[:, j] >= 0).flatten()
        r = rows[t, j].long()
        c, w, o = C[r].double(), weights[t, j].double()[:, None], go[t].double()
        out[t] += w * c
        size[t] += (w * c).abs()
        grad_C[r] = w * o
        grad_w[t, j] = (c * o).sum(1)
        size_w[t, j] = (c * o).abs().sum(1)
        del c, o
    got = fg.moe_combine(C, rows, weights).double()
    holds((got - out).abs(), (k + 1) * U * size * (1 + BF16) + BF16 * out.abs())
    del got, out, size
    keep = torch.full((M, N), 3.0, dtype=torch.bfloat16, device="cuda")
    got_C, got_w = fg.moe_combine_backward(go, C, rows, weights, grad_C=keep)
    holds((got_C.double() - grad_C).abs(), (BF16 + 2 * U) * grad_C.abs())
    holds((got_w.double() - grad_w).abs(), (N / 8 + 40) * U * size_w)
    assert bool((got_w[rows < 0] == 0).all())

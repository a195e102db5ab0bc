"""GPU tests of the operators around the GEMMs where values are lost first: infinities beside padded
ranks, products that all but cancel, softmax terms far below the largest, and loops that a CTA walks
many times.  Plain forms in float64 from the definitions in include/fp8gemm.h, on the device where
the sizes ask for it.

Tolerances: u = 2^-24 for each fp32 rounding, half a step of the output's type for the last one.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests import operators_reference as ref

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF16 = 2.0 ** -8  # half a step


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


# ------------------------------------------------------------------------------------- adapters
@pytest.mark.parametrize("M", [5, 40, 600])
@pytest.mark.parametrize("R", [8, 16, 24, 32, 40, 72, 96, 128])
def test_lora_infinite_rows_are_those_of_the_definition(fg, M, R):
    """A row with an infinity gives +inf, -inf or NaN where the definition does, at ranks that the kernels
    pad as at the others; the other rows hold what they held without it."""
    K, N, L = 144, 72, 2
    g = gen(M + R)
    C, x = torch.randn(M, N, generator=g).to(torch.bfloat16), torch.randn(M, K, generator=g).to(torch.bfloat16)
    a = (torch.rand(L, R, K, generator=g) + 0.5).to(torch.bfloat16)  # positive: h is +inf or -inf in whole
    b = (torch.rand(L, N, R, generator=g) + 0.5).to(torch.bfloat16)
    b[:, 1::3] *= -1
    b[:, 2::3, ::2] *= -1  # NaN: inf - inf
    ids = (torch.arange(M) % L).to(torch.int32)
    clean = fg.lora_add(C.cuda(), x.cuda(), a.cuda(), b.cuda(), ids.cuda()).cpu()
    x[1, 5], x[3, 100] = float("inf"), float("-inf")
    got = fg.lora_add(C.cuda(), x.cuda(), a.cuda(), b.cuda(), ids.cuda()).cpu()
    for m in (1, 3):
        with np.errstate(invalid="ignore"):
            want = f64(C[m]) + f64(b[m % L]) @ (f64(a[m % L]) @ f64(x[m]))
        want = np.where(np.arange(N) % 3 == 2, np.nan, want)  # (sums of both infinities, in any order)
        assert not np.isfinite(want).any()
        np.testing.assert_array_equal(f64(got[m]), want)
    keep = [m for m in range(M) if m not in (1, 3)]
    assert torch.equal(got[keep], clean[keep])


@pytest.mark.parametrize("M", [6, 700])
@pytest.mark.parametrize("R", [8, 16, 32, 64, 128])
def test_lora_sums_between_the_products_keep_fp32(fg, M, R):
    """Whole numbers below 2^24 throughout, so that fp32 sums are exact: C holds minus the rounded update, and what
    is left shows every bit of A x.  Exact, up to the one rounding of the output (no tolerance)."""
    K, N, L = 512, 136, 3
    g = gen(R + M)
    x = torch.randint(64, 128, (M, K), generator=g)
    a = torch.randint(0, 16, (L, R, K), generator=g)
    b = torch.randint(-1, 2, (L, N, R), generator=g) * (torch.rand(L, N, R, generator=g) < 8 / R)
    ids = torch.randint(0, L, (M,), generator=g)
    h = torch.stack([a[i] @ x[m] for m, i in enumerate(ids)])
    delta = torch.stack([b[i] @ h[m] for m, i in enumerate(ids)])
    most = torch.stack([b[i].abs() @ h[m] for m, i in enumerate(ids)])
    assert h.max() > 2 ** 18 and most.max() < 2 ** 24
    C = -delta.to(torch.bfloat16)
    want = (C.double() + delta.double()).to(torch.bfloat16)
    dev = [t.to(torch.bfloat16).cuda() for t in (C, x, a, b)]
    got = fg.lora_add(*dev, ids.to(torch.int32).cuda()).cpu()
    assert torch.equal(got, want)


@pytest.mark.parametrize("M", [4, 300])
@pytest.mark.parametrize("R", [8, 64])
def test_lora_sums_above_the_largest_bf16_stay_finite(fg, M, R):
    """A x = 1.9921875 2^127 + 2^119, an fp32 value that rounds to infinity in bf16; times 2^-120 it is 255.5, which is
    256 in bf16 (a tie to even)."""
    K, N = 32, 16
    x, a = torch.zeros(M, K), torch.zeros(1, R, K)
    x[:, 0], a[0, 1, 0] = 1.9921875 * 2.0 ** 64, 2.0 ** 63
    x[:, 17], a[0, 1, 17] = 2.0 ** 60, 2.0 ** 59
    b = torch.zeros(1, N, R)
    b[0, :, 1] = 2.0 ** -120
    dev = [t.to(torch.bfloat16).cuda() for t in (torch.zeros(M, N), x, a, b)]
    out = fg.lora_add(*dev, torch.zeros(M, dtype=torch.int32, device="cuda"))
    assert bool((out == 256.0).all())


# ------------------------------------------------------------------------------------- the router
@pytest.mark.parametrize("E", [9, 60, 100, 200, 400, 1000])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_weights_far_below_the_largest_logit(fg, E, renorm):
    """Logits in eighths, whose differences are exact: a weight is off by the roundings of e^d (2 ulp, 4 u), of the
    sum (40 u) and of the product (2 u), however far d is below 0; below the normal numbers by half a step
    of 2^-149 (2 ulp there: 2^-148)."""
    g = gen(E)
    T, k = 40, min(E, 32)
    logits = -torch.arange(E).float()[None] * 8.25 / min(E, 13) - torch.randint(0, 8, (T, E), generator=g) / 8
    logits[:, 3::4] -= 60.0
    logits = (logits * 8).round() / 8
    logits = logits.clamp(min=-104.0)
    logits[:, 0] = 0.0
    logits[0, 1:] = -90.125  # subnormal in every place but one
    want = ref.route(f64(logits)[None], k, None, renorm)
    ids, weights, _, _, _ = fg.moe_route(logits.cuda(), k, renormalize=renorm)
    assert np.array_equal(ids.cpu().numpy(), want["ids"][0])
    w = want["weights"][0]
    assert np.all(np.abs(f64(weights) - w) <= 48 * U * w + 2.0 ** -147)


@pytest.mark.parametrize("E", [9, 60, 200, 400])
def test_route_gradient_far_below_the_largest_logit(fg, E):
    """grad = p (h - sum p h): p carries 48 u as above, the bracket one rounding per term and sum."""
    T, k = 17, 2
    logits = -(torch.arange(T * E).view(T, E) % 700).float() / 8
    logits[:, 0], logits[:, 1] = 0.0, -0.125
    ids, weights, _, loss, slope = fg.moe_route(logits.cuda(), k)
    want = ref.route(f64(logits)[None], k)
    assert np.array_equal(ids.cpu().numpy(), want["ids"][0])
    gl = torch.tensor(3.0)
    got = f64(fg.moe_route_backward(logits.cuda(), ids, slope, None, gl.cuda()))
    grad, _ = ref.route_backward(want, None, f64(gl)[None])
    h = 3.0 * want["slope"][0]
    size = want["p"][0] * (h[None] + (want["p"][0] * h).sum(1, keepdims=True))
    # both sides' slope carries 4 u, the sum over E 40 u; below the normal numbers half steps of 2^-149
    assert np.all(np.abs(got - grad[0]) <= 110 * U * size + 2.0 ** -146 * (1 + h.max()))


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("T,E", [(40, 60), (5000, 256)])
def test_route_one_bad_logit_shows_in_its_sequence_alone(fg, T, E, bad):
    g = gen(T)
    logits = torch.randn(3, T, E, generator=g)
    clean = fg.moe_route(logits.cuda(), 3)
    want = fg.moe_route_backward(logits.cuda(), clean[0], clean[4], clean[1], torch.ones(3, device="cuda"))
    logits[1, 7, 11] = bad
    ids, weights, counts, loss, slope = fg.moe_route(logits.cuda(), 3)
    assert torch.isnan(loss).tolist() == [False, True, False]
    assert int(ids[1, 7, 0] == 11) == (bad == float("inf")) and len(set(ids[1, 7].tolist())) == 3
    got = fg.moe_route_backward(logits.cuda(), ids, slope, weights, torch.ones(3, device="cuda"))
    assert bool(got[1, 7].isnan().all()) and int(got.isnan().sum()) == E
    for s in (0, 2):
        assert torch.equal(ids[s], clean[0][s]) and torch.equal(got[s], want[s]) and torch.equal(loss[s], clean[3][s])
    assert torch.equal(weights[1, :7], clean[1][1, :7]) and torch.equal(weights[1, 8:], clean[1][1, 8:])


# ------------------------------------------------------------------------------------- dispatch
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_dispatch_over_all_exponents(fg, fmt):
    """The codes and scales of the cast alone, bit for bit, for rows whose largest values run over every exponent of
    bf16, below the normal numbers too, and whose others lie up to 2^-30 below."""
    g = gen(5)
    T, K = 1024, 256
    x = torch.randn(T, K, generator=g).abs().clamp(min=2.0 ** -9) * torch.exp2(-30 * torch.rand(T, K, generator=g) ** 3)
    x *= torch.where(torch.rand(T, K, generator=g) < 0.5, -1.0, 1.0)
    x[:, 5::16] = -0.0
    x = (x.double() * torch.exp2(torch.arange(T) % 262 - 136.0).double()[:, None]).clamp(-3.3e38, 3.3e38).to(torch.bfloat16).cuda()
    rows = torch.randperm(2 * T, generator=g).view(T, 2).to(torch.int32).cuda()
    A, sfa = fg.moe_dispatch_fp8(x, rows, shape=2 * T, fmt=fmt)
    q, s = fg.cast_fp8_rows(x, fmt=fmt)
    for j in range(2):
        at = rows[:, j].long()
        assert torch.equal(A[at], q) and torch.equal(sfa[:, at], s[:, :T])

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

"""The adapters' timeout on the GPU, without a fault: the products' thread of each kernel for many rows is made
to wait for a product that it has not issued (fg_lora_debug_set_stall).  The wait runs out after about two
seconds, the rows with an adapter are NaN, lora_status reports it, and the next call gives the bits of
the one before."""
from __future__ import annotations

import time

import pytest
import torch

pytestmark = pytest.mark.gpu

FG_ERR_TIMEOUT = 6


@pytest.mark.parametrize("R", [16, 64, 128])
@pytest.mark.parametrize("kernel", [1, 2])
def test_a_wait_that_runs_out_writes_nan(kernel, R):
    import moe_grouped_gemm_08_b200 as fg
    torch.cuda.set_device(0)
    g = torch.Generator().manual_seed(R)
    M, K, N, L = 2000, 1040, 1032, 5
    C, x, a, b = (torch.randn(*s, generator=g).to(torch.bfloat16).cuda() for s in ((M, N), (M, K), (L, R, K), (L, N, R)))
    ids = torch.randint(-1, L, (M,), generator=g).to(torch.int32).cuda()
    before = fg.lora_add(C, x, a, b, ids)
    assert fg.lora_status() == 0 and bool(before.isfinite().all())
    assert fg.lib.fg_lora_debug_set_stall(kernel) == 0
    try:
        t0 = time.time()
        out = fg.lora_add(C, x, a, b, ids)
        status = fg.lora_status()
        elapsed = time.time() - t0
    finally:
        assert fg.lib.fg_lora_debug_set_stall(0) == kernel
    assert status == FG_ERR_TIMEOUT and 1.0 < elapsed < 20.0
    assert bool(out[ids >= 0].isnan().all())
    assert torch.equal(out[ids < 0], C[ids < 0])
    assert fg.lora_status() == 0
    assert torch.equal(fg.lora_add(C, x, a, b, ids), before)
    assert fg.lora_status() == 0

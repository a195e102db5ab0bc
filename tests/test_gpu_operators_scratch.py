"""Missing or short scratch is refused on the host, before anything is launched."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

FG_ERR_INVALID_ARG, FG_ERR_ALIGNMENT = 1, 2


@pytest.fixture(scope="module")
def fg():
    import moe_grouped_gemm_08_b200 as lib
    torch.cuda.set_device(0)
    lib.init(0)
    return lib


def refusals(call, need, outputs):
    """`call(scratch address, bytes)` fails with none, with one byte too few and off its alignment, writing nothing; it
    works with `need` bytes."""
    assert need > 0
    scratch = torch.empty(need + 64, dtype=torch.uint8, device="cuda")
    before = [o.clone() for o in outputs]
    assert call(None, 0) == FG_ERR_INVALID_ARG
    assert call(None, need) == FG_ERR_INVALID_ARG
    assert call(scratch.data_ptr(), need - 1) == FG_ERR_INVALID_ARG
    assert call(scratch.data_ptr() + 2, need) == FG_ERR_ALIGNMENT
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(before, outputs))
    assert call(scratch.data_ptr(), need) == 0
    torch.cuda.synchronize()
    assert not any(torch.equal(a, b) for a, b in zip(before, outputs))


def test_router(fg):
    S, T, E, k = 2, 5000, 64, 4
    logits = torch.randn(S, T, E, device="cuda")
    ids, counts = (torch.full(s, -9, dtype=torch.int32, device="cuda") for s in ((S, T, k), (S, E)))
    weights, loss, slope = (torch.full(s, -9.0, device="cuda") for s in ((S, T, k), (S,), (S, E)))
    at = [t.data_ptr() for t in (ids, weights, counts, loss, slope)]
    refusals(lambda scratch, n: fg.lib.fg_moe_route(logits.data_ptr(), 0, None, *at, S, T, E, k, 1, scratch, n, None),
             fg.lib.fg_moe_route_scratch_bytes(S, T, E), [ids, weights, counts, loss, slope])
    torch.cuda.synchronize()
    assert torch.equal(ids, fg.moe_route(logits, k)[0])


def test_layout(fg):
    pairs, E = 5000, 8
    ids = torch.randint(0, E, (pairs,), device="cuda", dtype=torch.int32)
    M = fg.moe_layout_rows(pairs, E)
    rows, group = (torch.full((n,), -9, dtype=torch.int32, device="cuda") for n in (pairs, M))
    need = fg.lib.fg_moe_layout_scratch_bytes(pairs, E)
    refusals(lambda scratch, n: fg.lib.fg_moe_layout_contiguous(ids.data_ptr(), rows.data_ptr(), group.data_ptr(), pairs, E, M,
                                                                scratch, n, None), need, [rows, group])


@pytest.mark.parametrize("R", [16, 128])
def test_adapters(fg, R):
    M, N, K, L = 300, 72, 80, 3
    C, x, a, b = (torch.randn(*s, device="cuda").to(torch.bfloat16) for s in ((M, N), (M, K), (L, R, K), (L, N, R)))
    ids = torch.randint(0, L, (M,), device="cuda", dtype=torch.int32)
    out = torch.zeros_like(C)
    refusals(lambda scratch, n: fg.lib.fg_lora_add(C.data_ptr(), x.data_ptr(), a.data_ptr(), b.data_ptr(), ids.data_ptr(), None,
                                                   out.data_ptr(), M, N, K, R, L, scratch, n, None),
             fg.lib.fg_lora_scratch_bytes(M, R, L), [out])
    assert torch.equal(out, fg.lora_add(C, x, a, b, ids))

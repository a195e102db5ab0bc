"""The dispatch into float8 tensors, which the GEMMs take beside uint8 codes."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,dtype,other", [("e4m3", torch.float8_e4m3fn, torch.float8_e5m2),
                                             ("e5m2", torch.float8_e5m2, torch.float8_e4m3fn)])
def test_dispatch_into_float8(fmt, dtype, other):
    import moe_grouped_gemm_08_b200 as fg
    torch.cuda.set_device(0)
    fg.init(0)
    T, k, E, K, N = 20, 2, 3, 272, 136
    g = torch.Generator().manual_seed(1)
    x = torch.randn(T, K, generator=g).to(torch.bfloat16).cuda()
    B, sfb = fg.cast_fp8_blocks(torch.randn(E, N, K, generator=g).to(torch.bfloat16).cuda())
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).to(torch.int32).cuda()
    rows, group = fg.moe_layout_contiguous(ids, E)
    A = torch.zeros(group.numel(), K, dtype=torch.uint8, device="cuda")
    sfa = torch.zeros(-(-K // 128), fg.sfa_ld(group.numel()), device="cuda")
    fg.moe_dispatch_fp8(x, rows, A=A, sfa=sfa, fmt=fmt)
    A8, sfa8 = torch.zeros_like(A).view(dtype), torch.zeros_like(sfa)
    got, _ = fg.moe_dispatch_fp8(x, rows, A=A8, sfa=sfa8, fmt=fmt)
    assert got is A8 and torch.equal(A8.view(torch.uint8), A) and torch.equal(sfa8, sfa)
    C = fg.m_grouped_gemm_fp8_fp8_bf16_nt_contiguous(A8, sfa8, B, sfb, group)
    want = fg.m_grouped_gemm_fp8_fp8_bf16_nt_contiguous(A.view(dtype), sfa, B, sfb, group)
    held = rows.flatten().long()
    assert torch.equal(C[held], want[held])
    for wrong in (other, torch.int8, torch.float16):
        with pytest.raises(TypeError, match="A must"):
            fg.moe_dispatch_fp8(x, rows, A=torch.zeros(A.shape, dtype=wrong, device="cuda"), sfa=sfa, fmt=fmt)

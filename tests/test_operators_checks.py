"""CPU checks of the operators around the GEMMs: arguments are refused on the host, by the C ABI with
status codes and by the binding with exceptions, before anything is launched."""
from __future__ import annotations

import pytest
import torch

import moe_grouped_gemm_08_b200 as fg

NULL = None
P = 0x10000  # a fake aligned address: these calls fail (or do nothing) before any dereference
BIG = 1 << 40


def test_layout_rows_hold_every_choice():
    # the worst choice: every expert that has pairs has one more than a multiple of 128, or 1
    for pairs in (0, 1, 2, 127, 128, 129, 500, 1000, 5000):
        for E in (1, 2, 3, 8, 100):
            n = min(pairs, E)
            worst = 0
            if n:
                counts = [1] * n
                counts[0] += pairs - n
                worst = max(worst, sum(-(-c // 128) * 128 for c in counts))
                spread = [1 + 128 * ((pairs - n) // 128 // n)] * n
                if sum(spread) <= pairs:
                    worst = max(worst, sum(-(-c // 128) * 128 for c in spread))
            assert fg.moe_layout_rows(pairs, E) >= worst
            assert fg.moe_layout_rows(pairs, E) <= 128 * n + pairs


@pytest.mark.parametrize("change,expect", [
    (dict(), None), (dict(logits=NULL), 1), (dict(ids=NULL), 1), (dict(weights=NULL), 1), (dict(counts=NULL), 1),
    (dict(loss=NULL), 1), (dict(slope=NULL), 1), (dict(dtype=3), 1), (dict(S=-1), 1),
    (dict(T=-1), 1), (dict(E=0), 1), (dict(k=0), 1), (dict(k=9), 1), (dict(E=1025), 3), (dict(E=64, k=33), 3),
    (dict(S=65536), 3), (dict(logits=P + 2), 2), (dict(ids=P + 2), 2), (dict(S=0), 0),
])
def test_route_argument_errors(change, expect):
    a = dict(logits=P, dtype=0, mask=NULL, ids=P, weights=P, counts=P, loss=P, slope=P, S=1, T=4, E=8, k=2, renorm=1,
             scratch=P, bytes=0, stream=NULL)
    if expect is None:
        return
    a.update(change)
    assert fg.lib.fg_moe_route(*a.values()) == expect


@pytest.mark.parametrize("change,expect", [
    (dict(logits=NULL), 1), (dict(ids=NULL), 1), (dict(slope=NULL), 1), (dict(grad=NULL), 1), (dict(k=9), 1),
    (dict(dtype=-1), 1), (dict(E=1025), 3), (dict(grad=P + 1), 2), (dict(gw=P + 2), 2), (dict(S=0), 0), (dict(T=0), 0),
])
def test_route_backward_argument_errors(change, expect):
    a = dict(logits=P, dtype=1, ids=P, slope=P, gw=NULL, gl=NULL, grad=P, S=1, T=4, E=8, k=2, renorm=1, stream=NULL)
    a.update(change)
    assert fg.lib.fg_moe_route_backward(*a.values()) == expect


def test_layout_argument_errors():
    con, mas = fg.lib.fg_moe_layout_contiguous, fg.lib.fg_moe_layout_masked
    assert con(NULL, P, P, 10, 4, 512, NULL, 0, NULL) == 1
    assert con(P, P, NULL, 10, 4, 512, NULL, 0, NULL) == 1
    assert con(P, P, P, 10, 0, 512, NULL, 0, NULL) == 1
    assert con(P, P, P, -1, 4, 512, NULL, 0, NULL) == 1
    assert con(P, P, P, 10, 4, 511, NULL, 0, NULL) == 1      # fewer rows than a choice may take
    assert con(P, P, P, 10000, 4, 16384, NULL, 0, NULL) == 1  # scratch needed
    assert con(P, P, P, 10, 1025, BIG % (1 << 31), NULL, 0, NULL) == 3
    assert con(P, P, P, (1 << 24) + 1, 4, 1 << 26, P, BIG, NULL) == 3
    assert con(P + 2, P, P, 10, 4, 512, NULL, 0, NULL) == 2
    assert con(NULL, NULL, NULL, 0, 4, 0, NULL, 0, NULL) == 0
    assert mas(P, P, P, 10, 4, 0, NULL, 0, NULL) == 1
    assert mas(P, P, P, 10, 1024, 1 << 22, NULL, 0, NULL) == 3
    assert fg.lib.fg_moe_layout_scratch_bytes(2048, 8) == 0 < fg.lib.fg_moe_layout_scratch_bytes(2049, 8)


def test_dispatch_argument_errors():
    f = fg.lib.fg_moe_dispatch_fp8
    assert f(NULL, P, P, P, 4, 2, 1, 128, 256, 0, NULL) == 1
    assert f(P, P, P, P, 4, 2, 1, 128, 256, 2, NULL) == 1
    assert f(P, P, P, P, -1, 2, 1, 128, 256, 0, NULL) == 1
    assert f(P, P, P, P, 4, 2, 1, 128, 264, 0, NULL) == 2
    assert f(P + 8, P, P, P, 4, 2, 1, 128, 256, 0, NULL) == 2
    assert f(P, P, P + 8, P, 4, 2, 1, 128, 256, 0, NULL) == 2
    assert f(P, P, P, P, 4, 33, 1, 128, 256, 0, NULL) == 3
    assert f(P, P, P, P, 4, 2, 1 << 16, 1 << 15, 256, 0, NULL) == 3
    assert f(NULL, NULL, NULL, NULL, 0, 2, 1, 128, 256, 0, NULL) == 0
    assert f(NULL, NULL, NULL, NULL, 4, 0, 1, 128, 256, 0, NULL) == 0


def test_combine_argument_errors():
    f, b = fg.lib.fg_moe_combine, fg.lib.fg_moe_combine_backward
    assert f(NULL, P, P, P, 4, 2, 128, 64, NULL) == 1
    assert f(P, P, P, NULL, 4, 2, 128, 64, NULL) == 1
    assert f(P, P, P, P, 4, 2, 128, 60, NULL) == 2
    assert f(P + 8, P, P, P, 4, 2, 128, 64, NULL) == 2
    assert f(P, P, P, P, 4, 33, 128, 64, NULL) == 3
    assert f(NULL, NULL, NULL, NULL, 0, 2, 128, 64, NULL) == 0
    assert b(P, P, P, NULL, P, P, 4, 2, 128, 64, NULL) == 1
    assert b(P, P, P, P, P, NULL, 4, 2, 128, 64, NULL) == 1
    assert b(P, P, P, P, P + 8, P, 4, 2, 128, 64, NULL) == 2
    assert b(P, P, P, P, P, P, 4, 33, 128, 64, NULL) == 3
    assert b(P, P, P, P, P, P, 0, 2, 128, 64, NULL) == 0


@pytest.mark.parametrize("change,expect", [
    (dict(C=NULL), 1), (dict(x=NULL), 1), (dict(a=NULL), 1), (dict(b=NULL), 1), (dict(ids=NULL), 1), (dict(out=NULL), 1),
    (dict(M=-1), 1), (dict(L=-1), 1), (dict(K=24), 2), (dict(N=12), 2), (dict(R=12), 2), (dict(R=136), 3),
    (dict(x=P + 8), 2), (dict(out=P + 8), 2), (dict(scaling=P + 2), 2), (dict(M=0), 0), (dict(N=0), 0),
    (dict(M=(1 << 24) + 1), 3), (dict(M=(1 << 18) + 1, L=1024), 3), (dict(L=0, out=P, x=NULL, a=NULL, b=NULL), 0),
    (dict(R=0), 0), (dict(K=0), 0),
])
def test_lora_argument_errors(change, expect):
    a = dict(C=P, x=P, a=P, b=P, ids=P, scaling=NULL, out=P, M=4, N=64, K=64, R=16, L=2, scratch=NULL, bytes=0,
             stream=NULL)
    a.update(change)
    assert fg.lib.fg_lora_add(*a.values()) == expect


def test_binding_refuses_host_tensors_and_wrong_types():
    z = torch.zeros
    with pytest.raises(ValueError, match="CUDA"):
        fg.moe_route(z(4, 8), 2)
    with pytest.raises(TypeError, match="float32"):
        fg.moe_route(z(4, 8, dtype=torch.float64), 2)
    with pytest.raises(TypeError, match="ids"):
        fg.moe_layout_contiguous(z(4, 2, dtype=torch.int64), 8)
    with pytest.raises(TypeError, match="x must"):
        fg.moe_dispatch_fp8(z(4, 16, dtype=torch.bfloat16), z(4, 2, dtype=torch.int32), shape=128)
    with pytest.raises(TypeError, match="C must"):
        fg.moe_combine(z(4, 16, dtype=torch.bfloat16), z(4, 2, dtype=torch.int32))
    with pytest.raises(TypeError, match="C must"):
        fg.lora_add(z(4, 16), z(4, 16), z(1, 8, 16), z(1, 16, 8), z(4, dtype=torch.int32))
    with pytest.raises(ValueError, match="mmax"):
        fg.moe_layout_masked(z(4, 2, dtype=torch.int32), 8, 0)

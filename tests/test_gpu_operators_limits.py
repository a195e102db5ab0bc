"""GPU tests of the operators around the GEMMs at the top of the sizes that they accept: row and column
numbers next to 2^31.  Sums and values are chosen to be exact, so that nothing here has a tolerance
unless it says so."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu


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


@pytest.mark.parametrize("pairs", [10, 100_000])
def test_contiguous_layout_of_the_most_rows(fg, pairs):
    """m_indices of 2^31 - 1 rows, as the C ABI takes them: every row is written, and nothing in front."""
    M, E, front = 2 ** 31 - 1, 3, 1 << 23
    ids = torch.arange(pairs, device="cuda", dtype=torch.int32) % E
    rows = torch.empty_like(ids)
    buffer = torch.full((front + M,), 77, dtype=torch.int32, device="cuda")
    scratch = torch.empty(max(fg.lib.fg_moe_layout_scratch_bytes(pairs, E), 4), dtype=torch.uint8, device="cuda")
    code = fg.lib.fg_moe_layout_contiguous(ids.data_ptr(), rows.data_ptr(), buffer[front:].data_ptr(), pairs, E, M,
                                           scratch.data_ptr(), scratch.numel(), torch.cuda.current_stream().cuda_stream)
    assert code == 0
    torch.cuda.synchronize()
    want_rows, want = fg.moe_layout_contiguous(ids, E)
    assert torch.equal(rows, want_rows)
    assert bool((buffer[:front] == 77).all())
    group = buffer[front:]
    assert torch.equal(group[:want.numel()], want)
    assert bool((group[want.numel():] == -1).all())


@pytest.mark.parametrize("masked", [False, True])
def test_router_of_the_most_tokens(fg, masked):
    """2^31 - 1 tokens of one sequence and one expert: each takes it with weight 1, and its logit has no
    gradient.  (A chunk's sum of p holds at most 2^24 ones exactly; the sum of the chunks', eight per SM, and
    the division lose up to 1000 roundings of 2^-24.)"""
    T = 2 ** 31 - 1
    logits = torch.zeros(T, 1, dtype=torch.bfloat16, device="cuda")
    mask = None
    if masked:
        mask = torch.ones(T, dtype=torch.bool, device="cuda")
        mask[-1000:-1] = False
    routed = T - 999 * masked
    ids, weights, counts, loss, slope = fg.moe_route(logits, 1, mask=mask)
    assert counts.tolist() == [routed]
    assert abs(loss.item() - 1.0) <= 1000 * 2.0 ** -24
    assert abs(slope.item() * routed - 1.0) <= 4 * 2.0 ** -24
    for part, want in ((ids, 0), (weights, 1)):
        live, dead = (part[:T - 1000], part[T - 1000:T - 1]) if masked else (part, part[:0])
        assert bool((live == want).all()) and bool((part[-1:] == want).all())
        assert bool((dead == want - 1).all())  # id -1, weight 0
    del weights
    grad = fg.moe_route_backward(logits, ids, slope, None, torch.ones((), device="cuda"))
    assert not bool(grad.any())
    grad.fill_(1.0)
    del grad
    assert not bool(fg.moe_route_backward(logits, ids, slope, None, torch.ones((), device="cuda")).any())


@pytest.mark.parametrize("k", [1, 4, 5])
def test_combine_gradient_of_the_widest_rows(fg, k):
    """Rows of 2^31 - 8 columns, zero but for a few at both ends and between.  Every pass of the gradient's kernel over
    the columns (8192, 4096 or 2048 wide by k) ends at 2^31."""
    N = 2 ** 31 - 8
    at = torch.tensor([0, 7, 8191, 8192, 2 ** 30 + 5, N - 8193, N - 8184, N - 1], device="cuda")
    values = torch.arange(1, 9, device="cuda")
    C = torch.zeros(2, N, dtype=torch.bfloat16, device="cuda")
    C[1, at] = values.to(torch.bfloat16)
    grad_out = torch.zeros(1, N, dtype=torch.bfloat16, device="cuda")
    grad_out[0, at] = 2.0
    rows = torch.full((1, k), -1, dtype=torch.int32, device="cuda")
    rows[0, -1] = 1
    weights = torch.full((1, k), 0.5, device="cuda")
    grad_C = torch.full((2, N), 3.0, dtype=torch.bfloat16, device="cuda")
    _, grad_w = fg.moe_combine_backward(grad_out, C, rows, weights, grad_C=grad_C)
    assert grad_w[0].tolist() == [0.0] * (k - 1) + [72.0]
    assert bool((grad_C[0] == 3.0).all())
    assert bool((grad_C[1, at] == 1.0).all())
    grad_C[1, at] = 0.0
    assert not bool(grad_C[1].any())
    del grad_C, grad_out
    out = fg.moe_combine(C, rows, weights)
    assert torch.equal(out[0, at].float(), values * 0.5)
    out[0, at] = 0.0
    assert not bool(out.any())


def test_dispatch_of_the_widest_rows(fg):
    """Rows of 2^31 - 16 columns, the last block of them partial: codes and scales at both ends."""
    K = 2 ** 31 - 16
    x = torch.zeros(1, K, dtype=torch.bfloat16, device="cuda")
    x[0, 0], x[0, 1], x[0, K - 1], x[0, K - 2] = 448.0, -7.0, 896.0, 3.5
    rows = torch.tensor([[2, -1]], dtype=torch.int32, device="cuda")
    A = torch.full((4, K), 0xA5, dtype=torch.uint8, device="cuda")
    sfa = torch.full((2 ** 24, 4), -7.0, device="cuda")
    fg.moe_dispatch_fp8(x, rows, A=A, sfa=sfa)
    for other in (0, 1, 3):
        assert bool((A[other] == 0xA5).all()) and bool((sfa[:, other] == -7.0).all())
    codes = A[2].view(torch.float8_e4m3fn)
    assert codes[:2].float().tolist() == [448.0, -7.0] and codes[-2:].float().tolist() == [1.75, 448.0]
    assert int((A[2] != 0).sum()) == 4
    scale = sfa[:, 2]
    assert scale[0].item() == 1.0 and scale[-1].item() == 2.0 and bool((scale[1:-1] == 1.0).all())


def test_adapter_of_the_widest_rows(fg):
    """K = 2^31 - 16, then N = 2^31 - 8, the other small: few values beside zeros, at both ends."""
    K, N, R = 2 ** 31 - 16, 16, 8
    ids = torch.zeros(1, dtype=torch.int32, device="cuda")
    at = torch.tensor([0, 31, 32, 2 ** 30 + 3, K - 33, K - 1], device="cuda")
    x = torch.zeros(1, K, dtype=torch.bfloat16, device="cuda")
    x[0, at] = torch.arange(1.0, 7.0, device="cuda").to(torch.bfloat16)
    a = torch.zeros(1, R, K, dtype=torch.bfloat16, device="cuda")
    for r in range(R):
        a[0, r, at] = r + 1.0
    b = torch.zeros(1, N, R, dtype=torch.bfloat16, device="cuda")
    b[0, :, 0], b[0, 3, 7] = 1.0, 1.0
    C = torch.ones(1, N, dtype=torch.bfloat16, device="cuda")
    out = fg.lora_add(C, x, a, b, ids)[0]
    want = torch.full((N,), 22.0)
    want[3] += 168.0
    assert torch.equal(out.float().cpu(), want)
    del a, x
    N = 2 ** 31 - 8
    at = torch.tensor([0, 31, 32, 2 ** 30 + 3, N - 33, N - 1], device="cuda")
    b = torch.zeros(1, N, R, dtype=torch.bfloat16, device="cuda")
    b[0, at, 2] = torch.arange(1.0, 7.0, device="cuda").to(torch.bfloat16)
    x = torch.ones(1, 16, dtype=torch.bfloat16, device="cuda")
    a = torch.full((1, R, 16), 0.25, dtype=torch.bfloat16, device="cuda")
    C = torch.zeros(1, N, dtype=torch.bfloat16, device="cuda")
    out = fg.lora_add(C, x, a, b, ids)[0]
    assert out[at].tolist() == [4.0 * i for i in range(1, 7)]
    out[at] = 0.0
    assert not bool(out.any())


@pytest.mark.parametrize("T,E,k", [(2 ** 27, 16, 16), (2 ** 27 + 5, 32, 32)])
def test_balance_loss_of_more_choices_than_2_to_the_31(fg, T, E, k):
    """Every token takes every expert: an even load, whose loss is 1 and whose slope E f / n is 1 / n.  (p is 1 / E
    exactly; its sums over a chunk are exact, and the sum of eight chunks per SM loses up to 1300 u.)"""
    ids, weights, counts, loss, slope = fg.moe_route(torch.zeros(T, E, dtype=torch.bfloat16, device="cuda"), k)
    assert bool((ids == torch.arange(E, device="cuda", dtype=torch.int32)).all())
    assert bool((weights == 1.0 / E).all())
    assert counts.tolist() == [T] * E
    assert bool(((slope * T - 1.0).abs() <= 4 * 2.0 ** -24).all())
    assert abs(loss.item() - 1.0) <= 1300 * 2.0 ** -24

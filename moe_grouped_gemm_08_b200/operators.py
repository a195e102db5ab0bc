"""The operators around the grouped GEMMs: the router with its balance loss, the experts' row layout,
the cast into it, the weighted sum back, and low-rank adapters beside a projection.

  ids, weights, counts, loss, slope = moe_route(logits, top_k)          # forward
  rows, m_indices = moe_layout_contiguous(ids, E)                       # or moe_layout_masked
  A, sfa = moe_dispatch_fp8(x, rows, shape=m_indices.numel())           # FP8 rows of the experts
  C = m_grouped_gemm_fp8_fp8_bf16_nt_contiguous(A, sfa, B, sfb, m_indices)
  y = moe_combine(C, rows, weights)
  grad_logits = moe_route_backward(logits, ids, slope, grad_weights, grad_loss)
  lora_add(C, x, lora_a, lora_b, adapters, out=C)

Argument marshalling only, like the rest of the binding; gradients are explicit calls, as nothing
here takes part in autograd.  Outputs and scratch are allocated on the stream that the call runs on.
See include/fp8gemm.h for the definitions.
"""
from __future__ import annotations

import torch

from . import FORMATS, _bf16, _cdiv, _check, _f32, _i32, _lib, _stream

MAX_EXPERTS = 1024
DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


# Calls of a decode step are as long as their host side, so each entry point goes straight to the C
# ABI when it runs on the current device and stream, and otherwise once more with those made current.
_raw_stream = torch._C._cuda_getCurrentRawStream  # the handle without a Stream object


def _elsewhere(device, stream) -> bool:
    return stream is not None or device.index != torch.cuda.current_device()


def _there(device, stream, call, *args, **kwargs):
    """`call` with `device` and `stream` (None: the device's current one) current, so that what it
    allocates is not handed to another stream's work too early."""
    _stream(stream, device)  # checks that the stream is the device's
    with torch.cuda.device(device):
        if stream is None:
            return call(*args, **kwargs)
        with torch.cuda.stream(stream):
            return call(*args, **kwargs)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _logits(t: torch.Tensor):
    """(tensor, S, T, E) of router logits [T, E] or [S, T, E]."""
    if t.dtype not in DTYPES:
        raise TypeError(f"logits must be float32, bfloat16 or float16, got {t.dtype}")
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError("logits must be a contiguous CUDA tensor")
    if t.dim() not in (2, 3):
        raise ValueError("logits must be [T, E] or [S, T, E]")
    S, T, E = (1,) * (3 - t.dim()) + tuple(t.shape)
    return t, S, T, E


def _shaped(t: torch.Tensor, shape, what: str):
    if t.shape != shape:
        raise ValueError(f"{what} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t


def _same_device_as(first, **tensors):
    for name, t in tensors.items():
        if t is not None and t.get_device() != first.get_device():
            raise ValueError(f"{name} is on {t.device}, the first operand on {first.device}")


def _scratch(size, device):
    """(tensor or None, its address): scratch of a call, kept by the caller until it has launched."""
    if size == 0:
        return None, None
    t = torch.empty(size, dtype=torch.uint8, device=device)
    return t, t.data_ptr()


def _apart(out: torch.Tensor, what: str, **others):
    """`out` must not share memory with any of `others`."""
    a, b = out.data_ptr(), out.data_ptr() + out.numel() * out.element_size()
    for name, t in others.items():
        if t is not None and t.numel() and a < t.data_ptr() + t.numel() * t.element_size() and t.data_ptr() < b:
            raise ValueError(f"{what} must not overlap {name}")


# ------------------------------------------------------------------------------------- the router
def moe_route(logits, top_k, mask=None, renormalize=True, stream=None):
    """Top-k router with balance loss.  logits [T, E] or [S, T, E] (float32, bfloat16 or float16);
    mask [T] / [S, T] bool, False = a token that is not routed, whatever its logits hold.
    Returns (ids int32 [..., k], weights float32 [..., k], counts int32 [E] / [S, E], loss float32
    [] / [S], slope float32 [E] / [S, E]): choices in falling order (the lowest expert among equal
    logits; -1 with weight 0 for choices left over because logits are -inf or NaN), softmax weights,
    divided by their sum if `renormalize`, per-expert counts, one balance loss per sequence, and
    its derivative by the probabilities, which moe_route_backward takes."""
    logits, S, T, E = _logits(logits)
    k, lead, dev = int(top_k), logits.shape[:-2], logits.device
    if not 1 <= k <= E:
        raise ValueError(f"top_k must be in 1..{E}, got {k}")
    if mask is not None:
        if mask.dtype != torch.bool or not mask.is_cuda or not mask.is_contiguous():
            raise TypeError("mask must be a contiguous CUDA bool tensor")
        _shaped(mask, logits.shape[:-1], "mask")
        _same_device_as(logits, mask=mask)
    if _elsewhere(dev, stream):
        return _there(dev, stream, moe_route, logits, k, mask, renormalize)
    ids = torch.empty(logits.shape[:-1] + (k,), dtype=torch.int32, device=dev)
    weights = torch.empty_like(ids, dtype=torch.float32)
    counts = torch.empty(lead + (E,), dtype=torch.int32, device=dev)
    slope = torch.empty_like(counts, dtype=torch.float32)
    loss = torch.empty(lead, dtype=torch.float32, device=dev)
    size = _lib.fg_moe_route_scratch_bytes(S, T, E)
    scratch, at = _scratch(size, dev)
    _check(_lib.fg_moe_route(logits.data_ptr(), DTYPES[logits.dtype], _ptr(mask), ids.data_ptr(), weights.data_ptr(),
                             counts.data_ptr(), loss.data_ptr(), slope.data_ptr(), S, T, E, k, 1 if renormalize else 0,
                             at, size, _raw_stream(dev.index)), "fg_moe_route")
    return ids, weights, counts, loss, slope


def moe_route_backward(logits, ids, slope, grad_weights=None, grad_loss=None, renormalize=True, stream=None):
    """Gradient of moe_route's logits (same shape and type) from grad_weights float32 [..., k] and
    grad_loss float32 [] / [S], either None for none; ids and slope are the forward call's, and
    `renormalize` must be the same.  Zeros for tokens that were not routed."""
    logits, S, T, E = _logits(logits)
    ids, slope, dev = _i32(ids, "ids"), _f32(slope, "slope"), logits.device
    if ids.dim() != logits.dim() or ids.shape[:-1] != logits.shape[:-1]:
        raise ValueError("ids must be [..., k] beside logits [..., E]")
    _shaped(slope, logits.shape[:-2] + (E,), "slope")
    if grad_weights is not None:
        _shaped(_f32(grad_weights, "grad_weights"), ids.shape, "grad_weights")
    if grad_loss is not None:
        _shaped(_f32(grad_loss, "grad_loss"), logits.shape[:-2], "grad_loss")
    _same_device_as(logits, ids=ids, slope=slope, grad_weights=grad_weights, grad_loss=grad_loss)
    if _elsewhere(dev, stream):
        return _there(dev, stream, moe_route_backward, logits, ids, slope, grad_weights, grad_loss, renormalize)
    grad = torch.empty_like(logits)
    _check(_lib.fg_moe_route_backward(logits.data_ptr(), DTYPES[logits.dtype], ids.data_ptr(), slope.data_ptr(),
                                      _ptr(grad_weights), _ptr(grad_loss), grad.data_ptr(), S, T, E, ids.shape[-1],
                                      1 if renormalize else 0, _raw_stream(dev.index)), "fg_moe_route_backward")
    return grad


# ------------------------------------------------------------------------------------- row layouts
def moe_layout_rows(pairs, num_experts) -> int:
    """Rows of a contiguous layout that hold any choice of `pairs` (token, choice) pairs."""
    return int(_lib.fg_moe_layout_rows(int(pairs), int(num_experts)))


def _layout(ids, num_experts, mmax):
    """moe_layout_contiguous (mmax = 0) and moe_layout_masked on the current device and stream."""
    E, pairs = int(num_experts), ids.numel()
    rows = torch.empty_like(ids)
    size = _lib.fg_moe_layout_scratch_bytes(pairs, E)
    scratch, at = _scratch(size, ids.device)
    n = E if mmax else _lib.fg_moe_layout_rows(pairs, E)
    group = torch.empty(n, dtype=torch.int32, device=ids.device)
    call = _lib.fg_moe_layout_masked if mmax else _lib.fg_moe_layout_contiguous
    _check(call(ids.data_ptr(), rows.data_ptr(), group.data_ptr(), pairs, E, mmax or n, at, size,
                _raw_stream(ids.device.index)), "fg_moe_layout_masked" if mmax else "fg_moe_layout_contiguous")
    return rows, group


def _experts(num_experts):
    if not 1 <= num_experts <= MAX_EXPERTS:
        raise ValueError(f"num_experts must be in 1..{MAX_EXPERTS}, got {num_experts}")


def moe_layout_contiguous(ids, num_experts, stream=None):
    """Rows of each choice in the contiguous layout.  ids int32 [T, k] (any shape): the choice's
    expert, any value outside [0, num_experts) = none.  Returns (rows int32 like ids, -1 for none;
    m_indices int32 [M]) with M = moe_layout_rows(ids.numel(), num_experts), which no choice exceeds;
    an expert's rows are in the order of ids."""
    ids = _i32(ids, "ids")
    _experts(num_experts)
    if _elsewhere(ids.device, stream):
        return _there(ids.device, stream, _layout, ids, num_experts, 0)
    return _layout(ids, num_experts, 0)


def moe_layout_masked(ids, num_experts, mmax, stream=None):
    """Rows of each choice in the masked layout [num_experts, mmax] (expert * mmax + place), -1 for
    choices without an expert here and beyond the expert's mmax.  Returns (rows, masked_m)."""
    mmax = int(mmax)
    if mmax < 1:
        raise ValueError(f"mmax must be positive, got {mmax}")
    ids = _i32(ids, "ids")
    _experts(num_experts)
    if _elsewhere(ids.device, stream):
        return _there(ids.device, stream, _layout, ids, num_experts, mmax)
    return _layout(ids, num_experts, mmax)


def _rows(rows, tokens):
    rows = _i32(rows, "rows")
    if rows.dim() != 2 or rows.shape[0] != tokens:
        raise ValueError(f"rows must be [{tokens}, k], got {tuple(rows.shape)}")
    return rows


def moe_dispatch_fp8(x, rows, shape=None, A=None, sfa=None, fmt="e4m3", stream=None):
    """Cast x bf16 [T, K] into the experts' rows: the codes and scales of cast_fp8_rows(x[t]) at every
    row of rows[t] (int32 [T, k], from moe_layout_*).  `shape`: M for the contiguous layout, (G,
    Mmax) for the masked one; or give the outputs A uint8 [M, K] / [G, Mmax, K] and sfa.  Rows that
    no choice has are not written.  Returns (A, sfa)."""
    x = _bf16(x, "x")
    if x.dim() != 2:
        raise ValueError("x must be [T, K]")
    T, K = x.shape
    rows, dev = _rows(rows, T), x.device
    if (A is None) != (sfa is None) or (A is None and shape is None):
        raise ValueError("give shape, or both A and sfa")
    if A is not None:
        if A.dtype != torch.uint8 or not A.is_cuda or not A.is_contiguous() or A.dim() not in (2, 3):
            raise ValueError("A must be a contiguous CUDA uint8 tensor [M, K] or [G, Mmax, K]")
        if shape is not None and A.shape[:-1] != _lead(shape):
            raise ValueError("A does not have the given shape")
        shape = A.shape[:-1]
    shape = _lead(shape)
    G, M = shape if len(shape) == 2 else (1, *shape)
    scales = shape[:-1] + (_cdiv(K, 128), (M + 3) // 4 * 4)
    _same_device_as(x, rows=rows, A=A, sfa=sfa)
    if A is not None:
        _shaped(A, shape + (K,), "A")
        _shaped(_f32(sfa, "sfa"), scales, "sfa")
        _apart(A, "A", x=x, rows=rows, sfa=sfa)
        _apart(sfa, "sfa", x=x, rows=rows)
    if _elsewhere(dev, stream):
        return _there(dev, stream, moe_dispatch_fp8, x, rows, shape, A, sfa, fmt)
    if A is None:
        A = torch.empty(shape + (K,), dtype=torch.uint8, device=dev)
        sfa = torch.zeros(scales, dtype=torch.float32, device=dev)
    _check(_lib.fg_moe_dispatch_fp8(x.data_ptr(), rows.data_ptr(), A.data_ptr(), sfa.data_ptr(), T, rows.shape[1], G,
                                    M, K, FORMATS[fmt], _raw_stream(dev.index)), "fg_moe_dispatch_fp8")
    return A, sfa


def _lead(shape):
    return (int(shape),) if isinstance(shape, int) else tuple(int(n) for n in shape)


def _expert_rows(C, what):
    C = _bf16(C, what)
    if C.dim() not in (2, 3):
        raise ValueError(f"{what} must be [M, N] or [G, Mmax, N]")
    N = C.shape[-1]
    M = C.shape[0] if C.dim() == 2 else C.shape[0] * C.shape[1]
    if M > 0x7FFFFFFF:
        raise ValueError(f"{what} has too many rows")
    return C, M, N


def moe_combine(C, rows, weights=None, out=None, stream=None):
    """out[t] = sum_j weights[t, j] * C[rows[t, j]], bf16 [T, N], summed in float32; C bf16 [M, N] or
    [G, Mmax, N], rows int32 [T, k] with -1 for none, weights float32 [T, k] (None: all 1, the gradient
    of the dispatch)."""
    C, M, N = _expert_rows(C, "C")
    rows, dev = _rows(rows, rows.shape[0]), C.device
    T, k = rows.shape
    if weights is not None:
        _shaped(_f32(weights, "weights"), rows.shape, "weights")
    _same_device_as(C, rows=rows, weights=weights, out=out)
    if out is not None:
        _shaped(_bf16(out, "out"), (T, N), "out")
        _apart(out, "out", C=C, rows=rows, weights=weights)
    if _elsewhere(dev, stream):
        return _there(dev, stream, moe_combine, C, rows, weights, out)
    if out is None:
        out = torch.empty((T, N), dtype=torch.bfloat16, device=dev)
    _check(_lib.fg_moe_combine(C.data_ptr(), rows.data_ptr(), _ptr(weights), out.data_ptr(), T, k, M, N,
                               _raw_stream(dev.index)), "fg_moe_combine")
    return out


def moe_combine_backward(grad_out, C, rows, weights, grad_C=None, stream=None):
    """Gradients of moe_combine: (grad_C bf16 like C, grad_weights float32 [T, k]).  Rows of grad_C that
    no choice has are not written: give a zero-filled grad_C where they are read."""
    C, M, N = _expert_rows(C, "C")
    rows, dev = _rows(rows, rows.shape[0]), C.device
    T, k = rows.shape
    _shaped(_bf16(grad_out, "grad_out"), (T, N), "grad_out")
    _shaped(_f32(weights, "weights"), rows.shape, "weights")
    _same_device_as(C, rows=rows, weights=weights, grad_out=grad_out, grad_C=grad_C)
    if grad_C is not None:
        _shaped(_bf16(grad_C, "grad_C"), C.shape, "grad_C")
        _apart(grad_C, "grad_C", C=C, grad_out=grad_out, rows=rows, weights=weights)
    if _elsewhere(dev, stream):
        return _there(dev, stream, moe_combine_backward, grad_out, C, rows, weights, grad_C)
    if grad_C is None:
        grad_C = torch.empty_like(C)
    grad_weights = torch.empty_like(rows, dtype=torch.float32)
    _check(_lib.fg_moe_combine_backward(grad_out.data_ptr(), C.data_ptr(), rows.data_ptr(), weights.data_ptr(),
                                        grad_C.data_ptr(), grad_weights.data_ptr(), T, k, M, N,
                                        _raw_stream(dev.index)), "fg_moe_combine_backward")
    return grad_C, grad_weights


# ------------------------------------------------------------------------------------- adapters
def lora_add(C, x, lora_a, lora_b, adapters, scaling=None, out=None, stream=None):
    """out[m] = C[m] + scaling[a] * lora_b[a] @ (lora_a[a] @ x[m]) with a = adapters[m] (int32 [M]; any
    value outside [0, L) leaves C[m]).  C bf16 [M, N], x bf16 [M, K], lora_a bf16 [L, R, K], lora_b bf16
    [L, N, R], scaling float32 [L]; R a multiple of 8 up to 128.  out=C adds in place; None allocates."""
    C, x, lora_a, lora_b = _bf16(C, "C"), _bf16(x, "x"), _bf16(lora_a, "lora_a"), _bf16(lora_b, "lora_b")
    adapters, dev = _i32(adapters, "adapters"), C.device
    if C.dim() != 2 or x.dim() != 2 or lora_a.dim() != 3 or lora_b.dim() != 3:
        raise ValueError("inconsistent shapes")
    (M, N), K, (L, R) = C.shape, x.shape[1], lora_a.shape[:2]
    _shaped(x, (M, K), "x")
    _shaped(lora_a, (L, R, K), "lora_a")
    _shaped(lora_b, (L, N, R), "lora_b")
    _shaped(adapters, (M,), "adapters")
    if scaling is not None:
        _shaped(_f32(scaling, "scaling"), (L,), "scaling")
    _same_device_as(C, x=x, lora_a=lora_a, lora_b=lora_b, adapters=adapters, scaling=scaling, out=out)
    if out is not None:
        _shaped(_bf16(out, "out"), (M, N), "out")
        if out.data_ptr() != C.data_ptr():
            _apart(out, "out", C=C)
        _apart(out, "out", x=x, lora_a=lora_a, lora_b=lora_b, adapters=adapters, scaling=scaling)
    if _elsewhere(dev, stream):
        return _there(dev, stream, lora_add, C, x, lora_a, lora_b, adapters, scaling, out)
    if out is None:
        out = torch.empty_like(C)
    size = _lib.fg_lora_scratch_bytes(M, L)
    scratch, at = _scratch(size, dev)
    _check(_lib.fg_lora_add(C.data_ptr(), x.data_ptr(), lora_a.data_ptr(), lora_b.data_ptr(), adapters.data_ptr(),
                            _ptr(scaling), out.data_ptr(), M, N, K, R, L, at, size, _raw_stream(dev.index)),
           "fg_lora_add")
    return out


def lora_status(stream=None) -> int:
    """Synchronise the stream, then read and clear the status of lora_add on the current device: 0, or
    6 (FG_ERR_TIMEOUT) if a wait of one of its kernels has run out since the last read."""
    return int(_lib.fg_lora_status(_stream(stream)))

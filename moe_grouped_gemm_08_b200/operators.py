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

from . import FORMATS, _check, _lib, _stream

MAX_EXPERTS = 1024
DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}

# A call of a decode step takes as long as its host side does.  So each entry point goes straight to the C
# ABI when it runs on the current device and stream, and otherwise once more with those made current,
# and the checks below touch each tensor's attributes once.
_raw_stream = torch._C._cuda_getCurrentRawStream  # the handle, without a Stream object
_current_device = torch._C._cuda_getDevice


def _there(device, stream, call, *args):
    """`call` with `device` (an index) and `stream` (None: the device's current one) current, so that what
    it allocates is not handed to another stream's work too early."""
    _stream(stream, torch.device("cuda", device))  # checks that the stream is the device's
    with torch.cuda.device(device):
        if stream is None:
            return call(*args)
        with torch.cuda.stream(stream):
            return call(*args)


def _cuda(t, dtype, what):
    """A contiguous CUDA tensor of `dtype`; its device index."""
    if t.dtype is not dtype or not t.is_cuda or not t.is_contiguous():
        raise TypeError(f"{what} must be a contiguous CUDA {str(dtype)[6:]} tensor")
    return t.get_device()


def _beside(t, dtype, shape, device, what):
    """A contiguous tensor of `dtype` and `shape` on `device`; its address."""
    if t.dtype is not dtype or not t.is_contiguous():
        raise TypeError(f"{what} must be a contiguous CUDA {str(dtype)[6:]} tensor")
    if t.get_device() != device:
        raise ValueError(f"{what} is on {t.device}, the first operand on cuda:{device}")
    if t.shape != shape:
        raise ValueError(f"{what} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t.data_ptr()


def _apart(out: torch.Tensor, what: str, **others):
    """`out` must not share memory with any of `others`."""
    a = out.data_ptr()
    b = a + out.nbytes
    for name, t in others.items():
        if t is not None and t.data_ptr() < b and a < t.data_ptr() + t.nbytes and t.nbytes:
            raise ValueError(f"{what} must not overlap {name}")


def _scratch(size, like):
    """(tensor or None, its address): scratch of a call, kept by the caller until it has launched."""
    if size == 0:
        return None, None
    t = like.new_empty(size, dtype=torch.uint8)
    return t, t.data_ptr()


def _logits(t: torch.Tensor):
    """(type code, S, T, E, device index) of router logits [T, E] or [S, T, E]."""
    code = DTYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"logits must be float32, bfloat16 or float16, got {t.dtype}")
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError("logits must be a contiguous CUDA tensor")
    shape = t.shape
    if len(shape) == 3:
        return (code, *shape, t.get_device())
    if len(shape) != 2:
        raise ValueError("logits must be [T, E] or [S, T, E]")
    return (code, 1, *shape, t.get_device())


# ------------------------------------------------------------------------------------- the router
def moe_route(logits, top_k, mask=None, renormalize=True, stream=None):
    """Top-k router with balance loss.  logits [T, E] or [S, T, E] (float32, bfloat16 or float16);
    mask [T] / [S, T] bool, False = a token that is not routed, whatever its logits hold.
    Returns (ids int32 [..., k], weights float32 [..., k], counts int32 [E] / [S, E], loss float32
    [] / [S], slope float32 [E] / [S, E]): choices in falling order (the lowest expert among equal
    logits; -1 with weight 0 for choices left over because logits are -inf or NaN), softmax weights,
    divided by their sum if `renormalize`, per-expert counts, one balance loss per sequence, and
    its derivative by the probabilities, which moe_route_backward takes."""
    code, S, T, E, dev = _logits(logits)
    k, shape = int(top_k), logits.shape
    if not 1 <= k <= E:
        raise ValueError(f"top_k must be in 1..{E}, got {k}")
    mask_at = None if mask is None else _beside(mask, torch.bool, shape[:-1], dev, "mask")
    if stream is not None or dev != _current_device():
        return _there(dev, stream, moe_route, logits, k, mask, renormalize)
    ids = logits.new_empty(shape[:-1] + (k,), dtype=torch.int32)
    weights = torch.empty_like(ids, dtype=torch.float32)
    counts = logits.new_empty(shape[:-2] + (E,), dtype=torch.int32)
    slope = torch.empty_like(counts, dtype=torch.float32)
    loss = logits.new_empty(shape[:-2], dtype=torch.float32)
    size = _lib.fg_moe_route_scratch_bytes(S, T, E)
    scratch, at = _scratch(size, logits)
    _check(_lib.fg_moe_route(logits.data_ptr(), code, mask_at, ids.data_ptr(), weights.data_ptr(), counts.data_ptr(),
                             loss.data_ptr(), slope.data_ptr(), S, T, E, k, 1 if renormalize else 0, at, size,
                             _raw_stream(dev)), "fg_moe_route")
    return ids, weights, counts, loss, slope


def moe_route_backward(logits, ids, slope, grad_weights=None, grad_loss=None, renormalize=True, stream=None):
    """Gradient of moe_route's logits (same shape and type) from grad_weights float32 [..., k] and
    grad_loss float32 [] / [S], either None for none; ids and slope are the forward call's, and
    `renormalize` must be the same.  Zeros for tokens that were not routed."""
    code, S, T, E, dev = _logits(logits)
    shape = logits.shape
    if ids.dim() != len(shape) or ids.shape[:-1] != shape[:-1]:
        raise ValueError("ids must be [..., k] beside logits [..., E]")
    ids_at = _beside(ids, torch.int32, ids.shape, dev, "ids")
    slope_at = _beside(slope, torch.float32, shape[:-2] + (E,), dev, "slope")
    weights_at = loss_at = None
    if grad_weights is not None:
        weights_at = _beside(grad_weights, torch.float32, ids.shape, dev, "grad_weights")
    if grad_loss is not None:
        loss_at = _beside(grad_loss, torch.float32, shape[:-2], dev, "grad_loss")
    if stream is not None or dev != _current_device():
        return _there(dev, stream, moe_route_backward, logits, ids, slope, grad_weights, grad_loss, renormalize)
    grad = torch.empty_like(logits)
    _check(_lib.fg_moe_route_backward(logits.data_ptr(), code, ids_at, slope_at, weights_at, loss_at, grad.data_ptr(), S,
                                      T, E, ids.shape[-1], 1 if renormalize else 0, _raw_stream(dev)),
           "fg_moe_route_backward")
    return grad


# ------------------------------------------------------------------------------------- row layouts
def moe_layout_rows(pairs, num_experts) -> int:
    """Rows of a contiguous layout that hold any choice of `pairs` (token, choice) pairs."""
    return int(_lib.fg_moe_layout_rows(int(pairs), int(num_experts)))


def _layout(ids, num_experts, mmax, stream):
    """moe_layout_contiguous (mmax = 0) and moe_layout_masked."""
    E, dev, pairs = int(num_experts), _cuda(ids, torch.int32, "ids"), ids.numel()
    if not 1 <= E <= MAX_EXPERTS:
        raise ValueError(f"num_experts must be in 1..{MAX_EXPERTS}, got {E}")
    if stream is not None or dev != _current_device():
        return _there(dev, stream, _layout, ids, E, mmax, None)
    rows = torch.empty_like(ids)
    size = _lib.fg_moe_layout_scratch_bytes(pairs, E)
    scratch, at = _scratch(size, ids)
    if mmax:
        group = ids.new_empty(E)
        _check(_lib.fg_moe_layout_masked(ids.data_ptr(), rows.data_ptr(), group.data_ptr(), pairs, E, mmax, at, size,
                                         _raw_stream(dev)), "fg_moe_layout_masked")
    else:
        n = _lib.fg_moe_layout_rows(pairs, E)
        group = ids.new_empty(n)
        _check(_lib.fg_moe_layout_contiguous(ids.data_ptr(), rows.data_ptr(), group.data_ptr(), pairs, E, n, at, size,
                                             _raw_stream(dev)), "fg_moe_layout_contiguous")
    return rows, group


def moe_layout_contiguous(ids, num_experts, stream=None):
    """Rows of each choice in the contiguous layout.  ids int32 [T, k] (any shape): the choice's
    expert, any value outside [0, num_experts) = none.  Returns (rows int32 like ids, -1 for none;
    m_indices int32 [M]) with M = moe_layout_rows(ids.numel(), num_experts), which no choice exceeds;
    an expert's rows are in the order of ids."""
    return _layout(ids, num_experts, 0, stream)


def moe_layout_masked(ids, num_experts, mmax, stream=None):
    """Rows of each choice in the masked layout [num_experts, mmax] (expert * mmax + place), -1 for
    choices without an expert here and beyond the expert's mmax.  Returns (rows, masked_m)."""
    mmax = int(mmax)
    if mmax < 1:
        raise ValueError(f"mmax must be positive, got {mmax}")
    return _layout(ids, num_experts, mmax, stream)


def _rows(rows, tokens, device):
    """(k, address) of rows int32 [tokens, k]."""
    shape = rows.shape
    if len(shape) != 2 or shape[0] != tokens:
        raise ValueError(f"rows must be [{tokens}, k], got {tuple(shape)}")
    return shape[1], _beside(rows, torch.int32, shape, device, "rows")


def moe_dispatch_fp8(x, rows, shape=None, A=None, sfa=None, fmt="e4m3", stream=None):
    """Cast x bf16 [T, K] into the experts' rows: the codes and scales of cast_fp8_rows(x[t]) at every
    row of rows[t] (int32 [T, k], from moe_layout_*).  `shape`: M for the contiguous layout, (G,
    Mmax) for the masked one; or give the outputs A uint8 [M, K] / [G, Mmax, K] and sfa.  Rows that
    no choice has are not written.  Returns (A, sfa)."""
    dev = _cuda(x, torch.bfloat16, "x")
    if x.dim() != 2:
        raise ValueError("x must be [T, K]")
    T, K = x.shape
    k, rows_at = _rows(rows, T, dev)
    if (A is None) != (sfa is None) or (A is None and shape is None):
        raise ValueError("give shape, or both A and sfa")
    if A is not None:
        lead = A.shape[:-1]
        if shape is not None and lead != _lead(shape):
            raise ValueError("A does not have the given shape")
    else:
        lead = _lead(shape)
    if len(lead) not in (1, 2):
        raise ValueError("the layout is M rows or (G, Mmax)")
    G, M = lead if len(lead) == 2 else (1, lead[0])
    scales = lead[:-1] + ((K + 127) // 128, (M + 3) // 4 * 4)
    if A is not None:
        _beside(A, torch.uint8, lead + (K,), dev, "A")
        _beside(sfa, torch.float32, scales, dev, "sfa")
        _apart(A, "A", x=x, rows=rows, sfa=sfa)
        _apart(sfa, "sfa", x=x, rows=rows)
    if stream is not None or dev != _current_device():
        return _there(dev, stream, moe_dispatch_fp8, x, rows, lead, A, sfa, fmt)
    if A is None:
        A = x.new_empty(lead + (K,), dtype=torch.uint8)
        sfa = x.new_zeros(scales, dtype=torch.float32)
    _check(_lib.fg_moe_dispatch_fp8(x.data_ptr(), rows_at, A.data_ptr(), sfa.data_ptr(), T, k, G, M, K, FORMATS[fmt],
                                    _raw_stream(dev)), "fg_moe_dispatch_fp8")
    return A, sfa


def _lead(shape):
    return (shape,) if isinstance(shape, int) else tuple(int(n) for n in shape)


def _expert_rows(C):
    """(device index, M, N) of C bf16 [M, N] or [G, Mmax, N]."""
    dev, shape = _cuda(C, torch.bfloat16, "C"), C.shape
    if len(shape) not in (2, 3):
        raise ValueError("C must be [M, N] or [G, Mmax, N]")
    M = shape[0] if len(shape) == 2 else shape[0] * shape[1]
    if M > 0x7FFFFFFF:
        raise ValueError("C has too many rows")
    return dev, M, shape[-1]


def moe_combine(C, rows, weights=None, out=None, stream=None):
    """out[t] = sum_j weights[t, j] * C[rows[t, j]], bf16 [T, N], summed in float32; C bf16 [M, N] or
    [G, Mmax, N], rows int32 [T, k] with -1 for none, weights float32 [T, k] (None: all 1, the gradient
    of the dispatch)."""
    dev, M, N = _expert_rows(C)
    T = len(rows)
    k, rows_at = _rows(rows, T, dev)
    weights_at = None if weights is None else _beside(weights, torch.float32, rows.shape, dev, "weights")
    if out is not None:
        _beside(out, torch.bfloat16, (T, N), dev, "out")
        _apart(out, "out", C=C, rows=rows, weights=weights)
    if stream is not None or dev != _current_device():
        return _there(dev, stream, moe_combine, C, rows, weights, out)
    if out is None:
        out = C.new_empty((T, N))
    _check(_lib.fg_moe_combine(C.data_ptr(), rows_at, weights_at, out.data_ptr(), T, k, M, N, _raw_stream(dev)),
           "fg_moe_combine")
    return out


def moe_combine_backward(grad_out, C, rows, weights, grad_C=None, stream=None):
    """Gradients of moe_combine: (grad_C bf16 like C, grad_weights float32 [T, k]).  Rows of grad_C that
    no choice has are not written: give a zero-filled grad_C where they are read."""
    dev, M, N = _expert_rows(C)
    T = len(rows)
    k, rows_at = _rows(rows, T, dev)
    grad_out_at = _beside(grad_out, torch.bfloat16, (T, N), dev, "grad_out")
    weights_at = _beside(weights, torch.float32, rows.shape, dev, "weights")
    if grad_C is not None:
        _beside(grad_C, torch.bfloat16, C.shape, dev, "grad_C")
        _apart(grad_C, "grad_C", C=C, grad_out=grad_out, rows=rows, weights=weights)
    if stream is not None or dev != _current_device():
        return _there(dev, stream, moe_combine_backward, grad_out, C, rows, weights, grad_C)
    if grad_C is None:
        grad_C = torch.empty_like(C)
    grad_weights = torch.empty_like(weights)
    _check(_lib.fg_moe_combine_backward(grad_out_at, C.data_ptr(), rows_at, weights_at, grad_C.data_ptr(),
                                        grad_weights.data_ptr(), T, k, M, N, _raw_stream(dev)),
           "fg_moe_combine_backward")
    return grad_C, grad_weights


# ------------------------------------------------------------------------------------- adapters
def lora_add(C, x, lora_a, lora_b, adapters, scaling=None, out=None, stream=None):
    """out[m] = C[m] + scaling[a] * lora_b[a] @ (lora_a[a] @ x[m]) with a = adapters[m] (int32 [M]; any
    value outside [0, L) leaves C[m]).  C bf16 [M, N], x bf16 [M, K], lora_a bf16 [L, R, K], lora_b bf16
    [L, N, R], scaling float32 [L]; R a multiple of 8 up to 128.  out=C adds in place; None allocates."""
    dev = _cuda(C, torch.bfloat16, "C")
    if C.dim() != 2 or x.dim() != 2 or lora_a.dim() != 3:
        raise ValueError("C must be [M, N], x [M, K], lora_a [L, R, K]")
    (M, N), (L, R, K) = C.shape, lora_a.shape
    x_at = _beside(x, torch.bfloat16, (M, K), dev, "x")
    a_at = _beside(lora_a, torch.bfloat16, (L, R, K), dev, "lora_a")
    b_at = _beside(lora_b, torch.bfloat16, (L, N, R), dev, "lora_b")
    adapters_at = _beside(adapters, torch.int32, (M,), dev, "adapters")
    scaling_at = None if scaling is None else _beside(scaling, torch.float32, (L,), dev, "scaling")
    if out is not None:
        _beside(out, torch.bfloat16, (M, N), dev, "out")
        if out.data_ptr() != C.data_ptr():
            _apart(out, "out", C=C)
        _apart(out, "out", x=x, lora_a=lora_a, lora_b=lora_b, adapters=adapters, scaling=scaling)
    if stream is not None or dev != _current_device():
        return _there(dev, stream, lora_add, C, x, lora_a, lora_b, adapters, scaling, out)
    if out is None:
        out = torch.empty_like(C)
    size = _lib.fg_lora_scratch_bytes(M, R, L)
    scratch, at = _scratch(size, C)
    _check(_lib.fg_lora_add(C.data_ptr(), x_at, a_at, b_at, adapters_at, scaling_at, out.data_ptr(), M, N, K, R, L, at,
                            size, _raw_stream(dev)), "fg_lora_add")
    return out


def lora_status(stream=None) -> int:
    """Synchronise the stream, then read and clear the status of lora_add on the current device: 0, or
    6 (FG_ERR_TIMEOUT) if a wait of one of its kernels has run out since the last read."""
    return int(_lib.fg_lora_status(_stream(stream)))

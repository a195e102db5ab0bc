"""The operators around the grouped GEMMs: the router with its balance loss, the experts' row layout,
the cast into it, the weighted sum back, and low-rank adapters beside a projection.

  ids, weights, counts, loss, slope = moe_route(logits, top_k)          # forward
  rows, m_indices = moe_layout_contiguous(ids, E)                       # or moe_layout_masked
  A, sfa = moe_dispatch_fp8(x, rows, shape=m_indices.numel())           # FP8 rows of the experts
  C = m_grouped_gemm_fp8_fp8_bf16_nt_contiguous(A, sfa, B, sfb, m_indices)
  y = moe_combine(C, rows, weights)
  grad_logits = moe_route_backward(logits, ids, slope, grad_weights, grad_loss)
  lora_add(C, x, lora_a, lora_b, adapters, out=C)

Argument marshalling only, like the rest of the binding, and compiled (csrc/operators_binding.cpp), as a call
of a decode step takes as long as its host side.  Gradients are explicit calls: nothing here takes
part in autograd.  Outputs and scratch are allocated on the stream that the call runs on.  See
include/fp8gemm.h for the definitions.
"""
from __future__ import annotations

import torch

from . import FORMATS, FP8GemmError, _lib, _stream


class _Missing:
    """In the place of the compiled marshalling where it cannot be loaded: the GEMMs, which do without it, work, and
    the operators raise."""

    def __init__(self, why):
        self.why = why

    def __getattr__(self, name):
        raise ImportError(f"{name} needs {__package__}/_operators.so, which cannot be loaded ({self.why}); run "
                          "`python moe_grouped_gemm_08_b200/build.py` or __graft_entry__.build()")


try:
    from . import _operators
    _built_for = getattr(_operators, "torch_version", "another")
    if _built_for != torch.__version__:
        raise ImportError(f"built for torch {_built_for}, this is {torch.__version__}")
    _operators.set_error(FP8GemmError)
except ImportError as e:
    _operators = _Missing(e)


def _there(t, stream, call, *args):
    """`call` with t's device and `stream` (None: the device's current one) current, so that what it
    allocates is not handed to another stream's work too early."""
    _stream(stream, t.device)  # checks that the stream is the device's
    with torch.cuda.device(t.device):
        if stream is None:
            return call(*args)
        with torch.cuda.stream(stream):
            return call(*args)


def _call(t, stream, call, *args):
    """`call` on the current device and stream where those are meant; it answers None where t is on
    another device."""
    done = call(*args) if stream is None else None
    return _there(t, stream, call, *args) if done is None else done


# ------------------------------------------------------------------------------------- the router
def moe_route(logits, top_k, mask=None, renormalize=True, stream=None):
    """Top-k router with balance loss.  logits [T, E] or [S, T, E] (float32, bfloat16 or float16);
    mask [T] / [S, T] bool, False = a token that is not routed, whatever its logits hold.
    Returns (ids int32 [..., k], weights float32 [..., k], counts int32 [E] / [S, E], loss float32
    [] / [S], slope float32 [E] / [S, E]): choices in falling order (the lowest expert among equal
    logits; -1 with weight 0 for choices left over because logits are -inf or NaN), softmax weights,
    divided by their sum if `renormalize`, per-expert counts, one balance loss per sequence, and
    its derivative by the probabilities, which moe_route_backward takes."""
    return _call(logits, stream, _operators.moe_route, logits, top_k, mask, renormalize)


def moe_route_backward(logits, ids, slope, grad_weights=None, grad_loss=None, renormalize=True, stream=None):
    """Gradient of moe_route's logits (same shape and type) from grad_weights float32 [..., k] and
    grad_loss float32 [] / [S], either None for none; ids and slope are the forward call's, and
    `renormalize` must be the same.  Zeros for tokens that were not routed."""
    return _call(logits, stream, _operators.moe_route_backward, logits, ids, slope, grad_weights, grad_loss, renormalize)


# ------------------------------------------------------------------------------------- row layouts
def moe_layout_rows(pairs, num_experts) -> int:
    """Rows of a contiguous layout that hold any choice of `pairs` (token, choice) pairs."""
    return int(_lib.fg_moe_layout_rows(int(pairs), int(num_experts)))


def moe_layout_contiguous(ids, num_experts, stream=None):
    """Rows of each choice in the contiguous layout.  ids int32 [T, k] (any shape): the choice's
    expert, any value outside [0, num_experts) = none.  Returns (rows int32 like ids, -1 for none;
    m_indices int32 [M]) with M = moe_layout_rows(ids.numel(), num_experts), which no choice exceeds;
    an expert's rows are in the order of ids."""
    return _call(ids, stream, _operators.moe_layout, ids, num_experts, 0)


def moe_layout_masked(ids, num_experts, mmax, stream=None):
    """Rows of each choice in the masked layout [num_experts, mmax] (expert * mmax + place), -1 for
    choices without an expert here and beyond the expert's mmax.  Returns (rows, masked_m)."""
    if mmax < 1:
        raise ValueError(f"mmax must be positive, got {mmax}")
    return _call(ids, stream, _operators.moe_layout, ids, num_experts, mmax)


def moe_dispatch_fp8(x, rows, shape=None, A=None, sfa=None, fmt="e4m3", stream=None):
    """Cast x bf16 [T, K] into the experts' rows: the codes and scales of cast_fp8_rows(x[t]) at every
    row of rows[t] (int32 [T, k], from moe_layout_*).  `shape`: M for the contiguous layout, (G,
    Mmax) for the masked one; or give the outputs A [M, K] / [G, Mmax, K] (uint8, or the format's float8
    type) and sfa.  Rows that no choice has are not written.  Returns (A, sfa)."""
    if shape is not None:
        shape = (shape,) if isinstance(shape, int) else tuple(shape)
    return _call(x, stream, _operators.moe_dispatch_fp8, x, rows, shape, A, sfa, FORMATS[fmt])


def moe_combine(C, rows, weights=None, out=None, stream=None):
    """out[t] = sum_j weights[t, j] * C[rows[t, j]], bf16 [T, N], summed in float32; C bf16 [M, N] or
    [G, Mmax, N], rows int32 [T, k] with -1 for none, weights float32 [T, k] (None: all 1, the gradient
    of the dispatch)."""
    return _call(C, stream, _operators.moe_combine, C, rows, weights, out)


def moe_combine_backward(grad_out, C, rows, weights, grad_C=None, stream=None):
    """Gradients of moe_combine: (grad_C bf16 like C, grad_weights float32 [T, k]).  Rows of grad_C that
    no choice has are not written: give a zero-filled grad_C where they are read."""
    return _call(C, stream, _operators.moe_combine_backward, grad_out, C, rows, weights, grad_C)


# ------------------------------------------------------------------------------------- adapters
def lora_add(C, x, lora_a, lora_b, adapters, scaling=None, out=None, stream=None):
    """out[m] = C[m] + scaling[a] * lora_b[a] @ (lora_a[a] @ x[m]) with a = adapters[m] (int32 [M]; any
    value outside [0, L) leaves C[m]).  C bf16 [M, N], x bf16 [M, K], lora_a bf16 [L, R, K], lora_b bf16
    [L, N, R] (finite), scaling float32 [L]; R a multiple of 8 up to 128.  out=C adds in place; None allocates."""
    return _call(C, stream, _operators.lora_add, C, x, lora_a, lora_b, adapters, scaling, out)


def lora_status(stream=None) -> int:
    """Synchronise the stream, then read and clear the status of lora_add on the current device: 0, or
    6 (FG_ERR_TIMEOUT) if a wait of one of its kernels has run out since the last read."""
    return int(_lib.fg_lora_status(_stream(stream)))

"""Rotary tables, norm and turn, and block-sparse attention (include/svdq_attention.h): the
raw calls with the C names and argument order, and the tensor-level functions on top."""
from __future__ import annotations

import ctypes
from typing import Optional, Sequence

import torch

from ._binding import QkvEpilogue, qkv_epilogue
from ._tensors import (BF16, Entries, F32, I32T, I64, P, expect, on, one_device, ptr,
                       stream_ptr)

ROPE_MAX_AXES = 4


class RopeAxes(ctypes.Structure):
    """struct svdq_rope_axes of include/svdq_attention.h."""
    _fields_ = [("axes", ctypes.c_int32), ("dims", ctypes.c_int32 * ROPE_MAX_AXES),
                ("theta", ctypes.c_double * ROPE_MAX_AXES)]


_entries = Entries({
    "svdq_rope_tables": ([P, I64, ctypes.POINTER(RopeAxes), P, P, P], I32T),
    "svdq_qkv_norm_rope": ([P, I64, ctypes.POINTER(QkvEpilogue), P], I32T),
})
# Every symbol declared in include/svdq_attention.h.
EXPORTS_ATTENTION = _entries.names()


# ------------------------------------------------------------- raw C-ABI calls

def svdq_rope_tables(pos, S, axes: RopeAxes, cos_t, sin_t, stream=None):
    _entries.call("svdq_rope_tables", ptr(pos), S, ctypes.byref(axes), ptr(cos_t), ptr(sin_t),
                  stream_ptr(stream))


def svdq_qkv_norm_rope(qkv, M, epi: QkvEpilogue, stream=None):
    _entries.call("svdq_qkv_norm_rope", ptr(qkv), M, ctypes.byref(epi), stream_ptr(stream))


# ------------------------------------------------------------- tensor level

def rope_axes(dims: Sequence[int], theta=10000.0) -> RopeAxes:
    """How a head's dimension is divided among the axes; theta: one number, or one per axis."""
    dims = [int(d) for d in dims]
    if not 1 <= len(dims) <= ROPE_MAX_AXES:
        raise ValueError("1 to %d axes, got %d" % (ROPE_MAX_AXES, len(dims)))
    thetas = [float(theta)] * len(dims) if isinstance(theta, (int, float)) else \
        [float(t) for t in theta]
    if len(thetas) != len(dims):
        raise ValueError("%d dims and %d thetas" % (len(dims), len(thetas)))
    a = RopeAxes(axes=len(dims))
    for i, (d, t) in enumerate(zip(dims, thetas)):
        a.dims[i], a.theta[i] = d, t
    return a


def rope_tables(pos: torch.Tensor, dims: Sequence[int], theta=10000.0):
    """Positions fp32 [S, axes] -> (cos, sin) fp32 [S, sum(dims)/2], as linear_qkv and
    qkv_norm_rope take them.  Axis a turns dims[a] elements of each head; theta: one number,
    or one per axis."""
    axes = rope_axes(dims, theta)
    S = expect(pos, "pos", F32, (None, axes.axes)).shape[0]
    dev = one_device(pos=pos)
    t = torch.empty((2, S, sum(axes.dims) // 2), dtype=torch.float32, device=dev)
    cos_t, sin_t = t.unbind(0)
    with on(dev):
        svdq_rope_tables(pos, S, axes, cos_t, sin_t)
    return cos_t, sin_t


def qkv_norm_rope(qkv: torch.Tensor, heads: int, head_dim: int, seq: int, gamma_q, gamma_k,
                  eps: float, cos_t: torch.Tensor, sin_t: torch.Tensor):
    """A written projection bf16 [M, 3 heads head_dim] -> (Q, K, V) bf16 [M/seq, heads, seq,
    head_dim], Q and K with their RMS norm (gamma None: without) and rotary turn."""
    N = 3 * heads * head_dim
    M = expect(qkv, "qkv", BF16, (None, N)).shape[0]
    for what, g in (("gamma_q", gamma_q), ("gamma_k", gamma_k)):
        if g is not None:
            expect(g, what, BF16, (head_dim,))
    expect(cos_t, "cos_t", F32, (seq, head_dim // 2))
    expect(sin_t, "sin_t", F32, (seq, head_dim // 2))
    if seq < 1 or M % seq:
        raise ValueError("%d rows are no multiple of seq = %d" % (M, seq))
    dev = one_device(qkv=qkv, gamma_q=gamma_q, gamma_k=gamma_k, cos_t=cos_t, sin_t=sin_t)
    out = torch.empty((3, M // seq, heads, seq, head_dim), dtype=torch.bfloat16, device=dev)
    Q, K, V = out.unbind(0)
    epi = qkv_epilogue(heads, head_dim, seq, gamma_q, gamma_k, eps, cos_t, sin_t, Q, K, V)
    with on(dev):
        svdq_qkv_norm_rope(qkv, M, epi)
    return Q, K, V

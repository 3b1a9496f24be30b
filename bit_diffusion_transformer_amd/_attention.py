"""Rotary tables, norm and turn, and block-sparse attention (include/svdq_attention.h): the
raw calls with the C names and argument order, and the tensor-level functions on top."""
from __future__ import annotations

import ctypes
import functools
from typing import Optional, Sequence

import torch

from ._binding import QkvEpilogue
from ._tensors import (BF16, Entries, F32, F32T, I32, I32T, I64, P, SZ, at, expect, on,
                       one_device, ptr, scratch, stream_ptr)

ROPE_MAX_AXES = 4
QUERY_BLOCK, KEY_BLOCK = 128, 64


class RopeAxes(ctypes.Structure):
    """struct svdq_rope_axes of include/svdq_attention.h."""
    _fields_ = [("axes", ctypes.c_int32), ("dims", ctypes.c_int32 * ROPE_MAX_AXES),
                ("theta", ctypes.c_double * ROPE_MAX_AXES)]


class AttentionShape(ctypes.Structure):
    """struct svdq_attention_shape of include/svdq_attention.h."""
    _fields_ = [("batch", ctypes.c_int64), ("seq_q", ctypes.c_int64), ("seq_k", ctypes.c_int64),
                ("heads", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("keep", ctypes.c_int32), ("first", ctypes.c_int32)]


_SHAPE = ctypes.POINTER(AttentionShape)
_entries = Entries({
    "svdq_rope_tables": ([P, I64, ctypes.POINTER(RopeAxes), P, P, P], I32T),
    "svdq_qkv_norm_rope": ([P, I64, ctypes.POINTER(QkvEpilogue), P], I32T),
    "svdq_select_blocks_workspace_bytes": ([_SHAPE], SZ),
    "svdq_select_blocks": ([P, P, P, _SHAPE, P, P, SZ, P], I32T),
    "svdq_block_attention_workspace_bytes": ([_SHAPE], SZ),
    "svdq_block_attention": ([P, P, P, P, _SHAPE, F32T, P, P, P, SZ, P], I32T),
    "svdq_sparse_attention_workspace_bytes": ([_SHAPE], SZ),
    "svdq_sparse_attention": ([P, P, P, P, _SHAPE, F32T, P, P, P, SZ, P], I32T),
})
# Every symbol declared in include/svdq_attention.h.
EXPORTS_ATTENTION = _entries.names()


# ------------------------------------------------------------- raw C-ABI calls

def svdq_rope_tables(pos, S, axes: RopeAxes, cos_t, sin_t, stream=None):
    _entries.call("svdq_rope_tables", ptr(pos), S, ctypes.byref(axes), ptr(cos_t), ptr(sin_t),
                  stream_ptr(stream))


def svdq_qkv_norm_rope(qkv, M, epi: QkvEpilogue, stream=None):
    _entries.call("svdq_qkv_norm_rope", ptr(qkv), M, ctypes.byref(epi), stream_ptr(stream))


def svdq_select_blocks_workspace_bytes(shape: AttentionShape) -> int:
    return int(_entries["svdq_select_blocks_workspace_bytes"](ctypes.byref(shape)))


def svdq_select_blocks(q, k, kv_len, shape: AttentionShape, blocks, workspace, ws_bytes,
                       stream=None):
    _entries.call("svdq_select_blocks", ptr(q), ptr(k), ptr(kv_len), ctypes.byref(shape),
                  ptr(blocks), ptr(workspace), ws_bytes, stream_ptr(stream))


def svdq_block_attention_workspace_bytes(shape: AttentionShape) -> int:
    return int(_entries["svdq_block_attention_workspace_bytes"](ctypes.byref(shape)))


def svdq_block_attention(q, k, v, kv_len, shape: AttentionShape, scale, blocks, out, workspace,
                         ws_bytes, stream=None):
    _entries.call("svdq_block_attention", ptr(q), ptr(k), ptr(v), ptr(kv_len),
                  ctypes.byref(shape), scale, ptr(blocks), ptr(out), ptr(workspace), ws_bytes,
                  stream_ptr(stream))


def svdq_sparse_attention_workspace_bytes(shape: AttentionShape) -> int:
    return int(_entries["svdq_sparse_attention_workspace_bytes"](ctypes.byref(shape)))


def svdq_sparse_attention(q, k, v, kv_len, shape: AttentionShape, scale, blocks, out, workspace,
                          ws_bytes, stream=None):
    _entries.call("svdq_sparse_attention", ptr(q), ptr(k), ptr(v), ptr(kv_len),
                  ctypes.byref(shape), scale, ptr(blocks), ptr(out), ptr(workspace), ws_bytes,
                  stream_ptr(stream))


# ------------------------------------------------------------- tensor level

def _int32(n, what: str) -> int:
    """n as a C int32 (ctypes would drop higher bits silently)."""
    n = int(n)
    if not -2 ** 31 <= n < 2 ** 31:
        raise ValueError("%s: %d is out of range" % (what, n))
    return n


def rope_axes(dims: Sequence[int], theta=10000.0) -> RopeAxes:
    """How a head's dimension is divided among the axes; theta: one number, or one per axis."""
    dims = [_int32(d, "dims") for d in dims]
    if not 1 <= len(dims) <= ROPE_MAX_AXES:
        raise ValueError("1 to %d axes, got %d" % (ROPE_MAX_AXES, len(dims)))
    try:
        thetas = [float(theta)] * len(dims)
    except TypeError:
        thetas = [float(t) for t in theta]
    if len(thetas) != len(dims):
        raise ValueError("%d dims and %d thetas" % (len(dims), len(thetas)))
    a = RopeAxes(axes=len(dims))
    for i, (d, t) in enumerate(zip(dims, thetas)):
        a.dims[i], a.theta[i] = d, t
    return a


@functools.lru_cache(maxsize=64)
def _rope_division(dims, theta):
    """(RopeAxes, pairs of a token) of one division of the head: the same at every call."""
    axes = rope_axes(dims, theta)
    return axes, sum(axes.dims) // 2


def rope_tables(pos: torch.Tensor, dims: Sequence[int], theta=10000.0):
    """Positions fp32 [S, axes] -> (cos, sin) fp32 [S, sum(dims)/2], as linear_qkv and
    qkv_norm_rope take them.  Axis a turns dims[a] elements of each head; theta: one number,
    or one per axis."""
    dims = tuple(dims)
    if isinstance(theta, (int, float)):
        axes, pairs = _rope_division(dims, theta)
    else:
        axes = rope_axes(dims, theta)
        pairs = sum(axes.dims) // 2
    S = expect(pos, "pos", F32, (None, axes.axes))[0]
    dev = one_device(pos=pos)
    cos_t, sin_t = pos.new_empty((2, S, pairs)).unbind(0)
    with on(dev):
        _entries.call("svdq_rope_tables", at(pos), S, ctypes.byref(axes), at(cos_t), at(sin_t),
                      stream_ptr())
    return cos_t, sin_t


def qkv_norm_rope(qkv: torch.Tensor, heads: int, head_dim: int, seq: int, gamma_q, gamma_k,
                  eps: float, cos_t: torch.Tensor, sin_t: torch.Tensor):
    """A written projection bf16 [M, 3 heads head_dim] -> (Q, K, V) bf16 [M/seq, heads, seq,
    head_dim], Q and K with their RMS norm (gamma None: without) and rotary turn."""
    N = 3 * heads * head_dim
    M = expect(qkv, "qkv", BF16, (None, N))[0]
    for what, g in (("gamma_q", gamma_q), ("gamma_k", gamma_k)):
        if g is not None:
            expect(g, what, BF16, (head_dim,))
    expect(cos_t, "cos_t", F32, (seq, head_dim // 2))
    expect(sin_t, "sin_t", F32, (seq, head_dim // 2))
    if seq < 1 or M % seq:
        raise ValueError("%d rows are no multiple of seq = %d" % (M, seq))
    dev = one_device(qkv=qkv, gamma_q=gamma_q, gamma_k=gamma_k, cos_t=cos_t, sin_t=sin_t)
    out = qkv.new_empty((3, M // seq, heads, seq, head_dim), dtype=torch.bfloat16)
    Q, K, V = out.unbind(0)
    to, each = out.data_ptr(), M * heads * head_dim * 2
    epi = QkvEpilogue(heads, head_dim, seq, at(gamma_q), at(gamma_k), eps, at(cos_t),
                      at(sin_t), to, to + each, to + 2 * each)
    with on(dev):
        _entries.call("svdq_qkv_norm_rope", at(qkv), M, ctypes.byref(epi), stream_ptr())
    return Q, K, V


def _shape(q, k, kv_len, keep, first) -> AttentionShape:
    B, H, Sq, D = expect(q, "q", BF16, (None, None, None, None))
    _, G, Sk, _ = expect(k, "k", BF16, (B, None, None, D))
    if kv_len is not None:
        expect(kv_len, "kv_len", I32, (B,))
    return AttentionShape(B, Sq, Sk, H, G, D, _int32(keep, "keep"), _int32(first, "first"))


def _lists(s: AttentionShape):
    return (s.batch, s.heads, -(-s.seq_q // QUERY_BLOCK), s.keep)


def select_blocks(q, k, keep: int, first: int = 0, kv_len: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Q bf16 [B, H, Sq, D], K bf16 [B, G, Sk, D] -> int32 [B, H, ceil(Sq/128), keep]: for each
    block of 128 queries the `keep` blocks of 64 keys whose mean has the highest product with
    the queries' mean (the first `first` always), ascending, -1 behind the last."""
    s = _shape(q, k, kv_len, keep, first)
    dev = one_device(q=q, k=k, kv_len=kv_len)
    blocks = q.new_empty(_lists(s), dtype=torch.int32)
    need = svdq_select_blocks_workspace_bytes(s)
    ws = scratch(workspace, need, dev)
    with on(dev):
        _entries.call("svdq_select_blocks", at(q), at(k), at(kv_len), ctypes.byref(s), at(blocks),
                      at(ws), need, stream_ptr())
    return blocks


def block_attention(q, k, v, blocks, scale: Optional[float] = None,
                    kv_len: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Attention of each block of 128 queries over its list of key blocks (int32 [B, H,
    ceil(Sq/128), keep]) -> bf16 [B, Sq, H, D]; scale None: D^-1/2."""
    expect(blocks, "blocks", I32, (None, None, None, None))
    s = _shape(q, k, kv_len, blocks.shape[3], 0)
    expect(v, "v", BF16, tuple(k.shape))
    expect(blocks, "blocks", I32, _lists(s))
    dev = one_device(q=q, k=k, v=v, blocks=blocks, kv_len=kv_len)
    out = q.new_empty((s.batch, s.seq_q, s.heads, s.head_dim), dtype=torch.bfloat16)
    need = svdq_block_attention_workspace_bytes(s)
    ws = scratch(workspace, need, dev)
    with on(dev):
        _entries.call("svdq_block_attention", at(q), at(k), at(v), at(kv_len), ctypes.byref(s),
                      s.head_dim ** -0.5 if scale is None else scale, at(blocks), at(out), at(ws),
                      need, stream_ptr())
    return out


def sparse_attention(q, k, v, keep: int, first: int = 0, scale: Optional[float] = None,
                     kv_len: Optional[torch.Tensor] = None, return_blocks: bool = False,
                     workspace: Optional[torch.Tensor] = None):
    """select_blocks and block_attention in one call -> bf16 [B, Sq, H, D] (with the lists
    if return_blocks)."""
    s = _shape(q, k, kv_len, keep, first)
    expect(v, "v", BF16, tuple(k.shape))
    dev = one_device(q=q, k=k, v=v, kv_len=kv_len)
    out = q.new_empty((s.batch, s.seq_q, s.heads, s.head_dim), dtype=torch.bfloat16)
    blocks = q.new_empty(_lists(s), dtype=torch.int32) if return_blocks else None
    need = svdq_sparse_attention_workspace_bytes(s)
    ws = scratch(workspace, need, dev)
    with on(dev):
        _entries.call("svdq_sparse_attention", at(q), at(k), at(v), at(kv_len), ctypes.byref(s),
                      s.head_dim ** -0.5 if scale is None else scale, at(blocks), at(out), at(ws),
                      need, stream_ptr())
    return (out, blocks) if return_blocks else out

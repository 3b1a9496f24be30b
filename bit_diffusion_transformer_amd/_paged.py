"""Attention of packed sequences and over a paged cache, its page tables, and the norm and turn
that fills it (include/svdq_paged.h): the raw calls with the C names and argument order, and the
tensor-level functions on top."""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from ._tensors import (BF16, Entries, F32, F32T, I32, I32T, P, SZ, at, expect, expect_rows, on,
                       one_device, ptr, scratch, stream_of, stream_ptr)

MIN_PAGE, MAX_PAGE = 16, 256
MAX_SLOTS = 1 << 30


class PackedShape(ctypes.Structure):
    """struct svdq_packed_shape of include/svdq_paged.h."""
    _fields_ = [("tokens_q", ctypes.c_int64), ("tokens_k", ctypes.c_int64),
                ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64),
                ("v_stride", ctypes.c_int64), ("sequences", ctypes.c_int32),
                ("heads", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("causal", ctypes.c_int32)]


class PagedShape(ctypes.Structure):
    """struct svdq_paged_shape of include/svdq_paged.h."""
    _fields_ = [("tokens", ctypes.c_int64), ("pages", ctypes.c_int64), ("q_stride", ctypes.c_int64),
                ("requests", ctypes.c_int32), ("heads", ctypes.c_int32),
                ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("page", ctypes.c_int32),
                ("width", ctypes.c_int32), ("max_new", ctypes.c_int32), ("causal", ctypes.c_int32)]


class TableShape(ctypes.Structure):
    """struct svdq_table_shape of include/svdq_paged.h."""
    _fields_ = [("tokens", ctypes.c_int64), ("pages", ctypes.c_int64), ("free_count", ctypes.c_int64),
                ("requests", ctypes.c_int32), ("page", ctypes.c_int32), ("width", ctypes.c_int32)]


class CacheEpilogue(ctypes.Structure):
    """struct svdq_cache_epilogue of include/svdq_paged.h (device pointers as integers)."""
    _fields_ = [("tokens", ctypes.c_int64), ("table_rows", ctypes.c_int64), ("pages", ctypes.c_int64),
                ("heads", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("rotary", ctypes.c_int32), ("half", ctypes.c_int32),
                ("page", ctypes.c_int32), ("gamma_q", ctypes.c_void_p), ("gamma_k", ctypes.c_void_p),
                ("eps", ctypes.c_float), ("cos_t", ctypes.c_void_p), ("sin_t", ctypes.c_void_p),
                ("positions", ctypes.c_void_p), ("slots", ctypes.c_void_p), ("q", ctypes.c_void_p),
                ("k_cache", ctypes.c_void_p), ("v_cache", ctypes.c_void_p)]


_PACKED, _PAGED = ctypes.POINTER(PackedShape), ctypes.POINTER(PagedShape)
_entries = Entries({
    "svdq_packed_attention_workspace_bytes": ([_PACKED], SZ),
    "svdq_packed_attention": ([P, P, P, P, P, _PACKED, F32T, P, P, SZ, P], I32T),
    "svdq_paged_attention_workspace_bytes": ([_PAGED], SZ),
    "svdq_paged_attention": ([P, P, P, P, P, P, _PAGED, F32T, P, P, SZ, P], I32T),
    "svdq_page_tables": ([P, P, P, ctypes.POINTER(TableShape), P, P, P, P, P, P, P], I32T),
    "svdq_qkv_norm_rope_cache": ([P, ctypes.POINTER(CacheEpilogue), P], I32T),
})
# Every symbol declared in include/svdq_paged.h.
EXPORTS_PAGED = _entries.names()


# ------------------------------------------------------------- raw C-ABI calls
# q, k and v of the attentions may have rows further apart than their heads (the shape's
# strides say how far): their address alone is taken.

def svdq_packed_attention_workspace_bytes(shape: PackedShape) -> int:
    return int(_entries["svdq_packed_attention_workspace_bytes"](ctypes.byref(shape)))


def svdq_packed_attention(q, k, v, q_starts, k_starts, shape: PackedShape, scale, out, workspace,
                          ws_bytes, stream=None):
    _entries.call("svdq_packed_attention", at(q), at(k), at(v), ptr(q_starts), ptr(k_starts),
                  ctypes.byref(shape), scale, ptr(out), ptr(workspace), ws_bytes, stream_ptr(stream))


def svdq_paged_attention_workspace_bytes(shape: PagedShape) -> int:
    return int(_entries["svdq_paged_attention_workspace_bytes"](ctypes.byref(shape)))


def svdq_paged_attention(q, k_cache, v_cache, tables, q_starts, kv_len, shape: PagedShape, scale, out,
                         workspace, ws_bytes, stream=None):
    _entries.call("svdq_paged_attention", at(q), ptr(k_cache), ptr(v_cache), ptr(tables),
                  ptr(q_starts), ptr(kv_len), ctypes.byref(shape), scale, ptr(out), ptr(workspace),
                  ws_bytes, stream_ptr(stream))


def svdq_page_tables(cached, added, free_pages, shape: TableShape, tables, q_starts, kv_len, slots,
                     positions, counts, stream=None):
    _entries.call("svdq_page_tables", ptr(cached), ptr(added), ptr(free_pages), ctypes.byref(shape),
                  ptr(tables), ptr(q_starts), ptr(kv_len), ptr(slots), ptr(positions), ptr(counts),
                  stream_ptr(stream))


def svdq_qkv_norm_rope_cache(qkv, epi: CacheEpilogue, stream=None):
    _entries.call("svdq_qkv_norm_rope_cache", ptr(qkv), ctypes.byref(epi), stream_ptr(stream))


# ------------------------------------------------------------- tensor level

def _out(out: Optional[torch.Tensor], q: torch.Tensor, what: str = "out") -> torch.Tensor:
    """`out`, checked, or a new tensor of q's shape."""
    if out is None:
        if q.dtype is torch.bfloat16 and q.is_contiguous():
            return torch.empty_like(q)             # (half the time of the other)
        return torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
    expect(out, what, BF16, tuple(q.shape))
    return out


def _range(sizes: dict) -> None:
    """The error of sizes of which one is no C int32 (ctypes would drop its higher bits)."""
    raise ValueError("out of range: %s" % ", ".join("%s = %d" % x for x in sizes.items()))


def _scale(scale: Optional[float], D: int) -> float:
    return max(D, 1) ** -0.5 if scale is None else scale


def _max_new(max_new, tokens: int) -> int:
    """The most new tokens of a request: at most all of them."""
    if max_new is None:
        return max(tokens, 1)
    if max_new < 1:
        raise ValueError("max_new must be at least 1, got %d" % max_new)
    return min(max_new, max(tokens, 1))


def packed_attention(q, k, v, q_starts, k_starts: Optional[torch.Tensor] = None, causal: bool = True,
                     scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Attention of sequences packed one after another: q bf16 [T, H, D], k and v bf16 [Tk, G, D]
    (parts of one projection may be passed as they are), q_starts int32 [sequences + 1], k_starts
    likewise where the keys are others -> bf16 [T, H, D].  causal: a row sees the keys up to its
    own, the last row all.  scale None: D^-1/2.  Rows of no sequence are left as they were."""
    (T, H, D), qs = expect_rows(q, "q", BF16, (None, None, None))
    (Tk, G, _), ks = expect_rows(k, "k", BF16, (None, None, D))
    _, vs = expect_rows(v, "v", BF16, (Tk, G, D))
    B = expect(q_starts, "q_starts", I32, (None,))[0] - 1
    if B < 0:
        raise ValueError("q_starts: expected at least one entry")
    if (B | H | G | D) >> 31:
        _range(dict(sequences=B, heads=H, kv_heads=G, head_dim=D))
    if k_starts is not None:
        expect(k_starts, "k_starts", I32, (B + 1,))
    elif Tk != T:
        raise ValueError("k has %d rows, q %d: k_starts is needed" % (Tk, T))
    out = _out(out, q)
    dev = one_device(q=q, k=k, v=v, q_starts=q_starts, k_starts=k_starts, out=out)
    shape = PackedShape(T, Tk, qs, ks, vs, B, H, G, D, bool(causal))
    need = svdq_packed_attention_workspace_bytes(shape)
    ws = scratch(workspace, need, dev)
    with on(dev):
        _entries.call("svdq_packed_attention", at(q), at(k), at(v), at(q_starts), at(k_starts),
                      ctypes.byref(shape), _scale(scale, D), at(out), at(ws), need, stream_of(dev))
    return out


def paged_attention(q, k_cache, v_cache, tables, q_starts, kv_len, max_new: Optional[int] = None,
                    causal: bool = True, scale: Optional[float] = None,
                    out: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Attention of new tokens over a paged cache: q bf16 [T, H, D], caches bf16 [pages, G, page, D],
    tables int32 [requests, width] of page numbers, q_starts int32 [requests + 1], kv_len int32
    [requests] (the new tokens' keys, already in the cache, included) -> bf16 [T, H, D].  max_new:
    the most new tokens of a request, if known (1 when decoding, which is up to a fifth slower
    without it).  causal, scale and out as for packed_attention."""
    (T, H, D), qs = expect_rows(q, "q", BF16, (None, None, None))
    pages, G, page, _ = expect(k_cache, "k_cache", BF16, (None, None, None, D))
    expect(v_cache, "v_cache", BF16, (pages, G, page, D))
    B, width = expect(tables, "tables", I32, (None, None))
    expect(q_starts, "q_starts", I32, (B + 1,))
    expect(kv_len, "kv_len", I32, (B,))
    if (B | H | G | D | page | width) >> 31:
        _range(dict(requests=B, heads=H, kv_heads=G, head_dim=D, page=page, width=width))
    out = _out(out, q)
    dev = one_device(q=q, k_cache=k_cache, v_cache=v_cache, tables=tables, q_starts=q_starts,
                     kv_len=kv_len, out=out)
    shape = PagedShape(T, pages, qs, B, H, G, D, page, width, _max_new(max_new, T), bool(causal))
    need = svdq_paged_attention_workspace_bytes(shape)
    ws = scratch(workspace, need, dev)
    with on(dev):
        _entries.call("svdq_paged_attention", at(q), at(k_cache), at(v_cache), at(tables),
                      at(q_starts), at(kv_len), ctypes.byref(shape), _scale(scale, D), at(out),
                      at(ws), need, stream_of(dev))
    return out


def page_tables(cached, added, free_pages, tables, page: int, pages: int, tokens: int):
    """The page tables of a step: requests hold cached[b] tokens (int32 [requests]) and get
    added[b] more; the pages they lack are taken from free_pages (int32) in order and written into
    tables (int32 [requests, width], in place) -> (q_starts int32 [requests + 1], kv_len int32
    [requests], slots int32 [tokens], positions int32 [tokens], counts int32 [2]: pages taken, new
    tokens without a slot).  pages: the cache's; tokens: rows of the step, at least sum(added);
    rows behind the last request get slot and position -1."""
    B = expect(cached, "cached", I32, (None,))[0]
    expect(added, "added", I32, (B,))
    F = expect(free_pages, "free_pages", I32, (None,))[0]
    width = expect(tables, "tables", I32, (B, None))[1]
    if not 0 <= tokens < 1 << 31 or not 0 <= pages < 1 << 31 or not 0 < page <= MAX_PAGE:
        raise ValueError("page = %d, pages = %d, tokens = %d" % (page, pages, tokens))
    if (B | width) >> 31:
        _range(dict(requests=B, width=width))
    dev = one_device(cached=cached, added=added, free_pages=free_pages, tables=tables)
    q_starts, kv_len, slots, positions, counts = torch.split_with_sizes(
        cached.new_empty(2 * (B + tokens) + 3), (B + 1, B, tokens, tokens, 2))
    shape = TableShape(tokens, pages, F, B, page, width)
    with on(dev):
        _entries.call("svdq_page_tables", at(cached), at(added), at(free_pages), ctypes.byref(shape),
                      at(tables), at(q_starts), at(kv_len), at(slots), at(positions), at(counts),
                      stream_of(dev))
    return q_starts, kv_len, slots, positions, counts


def qkv_norm_rope_cache(qkv, heads: int, kv_heads: int, gamma_q, gamma_k, eps: float, cos_t, sin_t,
                        positions, slots, k_cache, v_cache, half: bool = False,
                        out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """A written projection bf16 [T, (heads + 2 kv_heads) D] with the RMS norm (gamma None:
    without) and rotary turn of Q and K -> Q bf16 [T, heads, D]; K and V go to the slots (int32
    [T]) of the caches bf16 [pages, kv_heads, page, D].  cos_t, sin_t fp32 [rows, rotary / 2], taken
    by positions (int32 [T]), turn the first `rotary` columns of each head: pairs of neighbours, or
    with `half` of the two halves.  A slot outside the cache: nothing is cached; a position outside
    the tables: that row is left as it was."""
    pages, G, page, D = expect(k_cache, "k_cache", BF16, (None, kv_heads, None, None))
    expect(v_cache, "v_cache", BF16, (pages, G, page, D))
    T = expect(qkv, "qkv", BF16, (None, (heads + 2 * kv_heads) * D))[0]
    for what, g in (("gamma_q", gamma_q), ("gamma_k", gamma_k)):
        if g is not None:
            expect(g, what, BF16, (D,))
    rows, pairs = expect(cos_t, "cos_t", F32, (None, None))
    expect(sin_t, "sin_t", F32, (rows, pairs))
    expect(positions, "positions", I32, (T,))
    expect(slots, "slots", I32, (T,))
    if (heads | kv_heads | D | 2 * pairs | page) >> 31:
        _range(dict(heads=heads, kv_heads=kv_heads, head_dim=D, rotary=2 * pairs, page=page))
    if out is None:
        out = torch.empty((T, heads, D), dtype=torch.bfloat16, device=qkv.device)
    else:
        expect(out, "out", BF16, (T, heads, D))
    dev = one_device(qkv=qkv, gamma_q=gamma_q, gamma_k=gamma_k, cos_t=cos_t, sin_t=sin_t,
                     positions=positions, slots=slots, k_cache=k_cache, v_cache=v_cache, out=out)
    epi = CacheEpilogue(T, rows, pages, heads, kv_heads, D, 2 * pairs, bool(half), page, at(gamma_q),
                        at(gamma_k), eps, at(cos_t), at(sin_t), at(positions), at(slots), at(out),
                        at(k_cache), at(v_cache))
    with on(dev):
        _entries.call("svdq_qkv_norm_rope_cache", at(qkv), ctypes.byref(epi), stream_of(dev))
    return out


class CacheStep:
    """qkv_norm_rope_cache and paged_attention of one layer's T rows, on tensors whose types, shapes
    and device fit together: what either would refuse is refused here, without a launch."""

    def __init__(self, T: int, heads: int, kv_heads: int, head_dim: int, gamma_q, gamma_k, eps: float, cos_t,
                 sin_t, positions, slots, k_cache, v_cache, tables, q_starts, kv_len, max_new, causal: bool,
                 half: bool):
        rows, pairs = cos_t.shape
        B, width = tables.shape
        pages, _, page, _ = k_cache.shape
        if (B | heads | kv_heads | head_dim | 2 * pairs | page | width) >> 31:
            _range(dict(requests=B, heads=heads, kv_heads=kv_heads, head_dim=head_dim, rotary=2 * pairs, page=page,
                        width=width))
        tabs = [at(cos_t), at(sin_t), at(positions), at(slots)]
        caches, lists = [at(k_cache), at(v_cache)], [at(tables), at(q_starts), at(kv_len)]
        gammas = [at(gamma_q), at(gamma_k)]
        self._q = (T, heads, head_dim)
        # (no tokens yet: the sizes are checked, the addresses are not)
        self._epi = CacheEpilogue(0, rows, pages, heads, kv_heads, head_dim, 2 * pairs, bool(half), page, *gammas,
                                  eps, *tabs, None, *caches)
        _entries.call("svdq_qkv_norm_rope_cache", None, ctypes.byref(self._epi), None)
        if (tabs[0] | tabs[1] | caches[0] | caches[1] | (gammas[0] or 0) | (gammas[1] or 0)) & 15 or (
                tabs[2] | tabs[3] | lists[0] | lists[1] | lists[2]) & 3:
            raise ValueError("the caches, the rotary tables and gamma must be 16-byte aligned, lengths "
                             "and tables 4-byte")
        self._shape = PagedShape(T, pages, heads * head_dim, B, heads, kv_heads, head_dim, page, width,
                                 _max_new(max_new, T), bool(causal))
        self._need = svdq_paged_attention_workspace_bytes(self._shape)
        self._rest = [*caches, *lists, ctypes.byref(self._shape), _scale(None, head_dim)]
        if self._need == 0 and T and B:            # refused for its sizes, whatever the tensors
            _entries.call("svdq_paged_attention", None, *self._rest, None, None, 0, None)

    def run(self, qkv: torch.Tensor) -> torch.Tensor:
        """A projection bf16 [T, (heads + 2 kv_heads) head_dim] on the current device -> the
        attention's rows bf16 [T, heads, head_dim]; its keys and values are in the caches then."""
        q, out = torch.empty((2,) + self._q, dtype=torch.bfloat16, device=qkv.device)
        ws = scratch(None, self._need, qkv.device)
        stream = stream_of(qkv.device)
        self._epi.tokens, self._epi.q = self._q[0], at(q)
        _entries.call("svdq_qkv_norm_rope_cache", at(qkv), ctypes.byref(self._epi), stream)
        _entries.call("svdq_paged_attention", at(q), *self._rest, at(out), at(ws), self._need, stream)
        return out

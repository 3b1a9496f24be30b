"""The 8-bit integer linear (include/svdq_i8.h): the raw calls with the C names and argument
order, and the tensor-level functions on top."""
from __future__ import annotations

from typing import Optional

import torch

from ._binding import ACT_NONE
from ._tensors import (BF16, Entries, F32, I32T, I64, I8, P, SZ, at, expect, on, one_device,
                       ptr, scratch, stream_ptr)

_entries = Entries({
    "svdq_i8_pack_weights": ([P, I64, I64, P, P, P], I32T),
    "svdq_i8_quantize_act": ([P, P, I64, I64, P, P, P], I32T),
    "svdq_i8_gemm_workspace_bytes": ([I64, I64, I64], SZ),
    "svdq_i8_gemm": ([P, P, P, P, P, I32T, I64, I64, I64, P, P, SZ, P], I32T),
    "svdq_i8_linear_workspace_bytes": ([I64, I64, I64], SZ),
    "svdq_i8_linear": ([P, P, P, P, P, I32T, I64, I64, I64, P, P, SZ, P], I32T),
})
# Every symbol declared in include/svdq_i8.h.
EXPORTS_I8 = _entries.names()


# ------------------------------------------------------------- raw C-ABI calls

def svdq_i8_pack_weights(W, N, K, qw, sw, stream=None):
    _entries.call("svdq_i8_pack_weights", ptr(W), N, K, ptr(qw), ptr(sw), stream_ptr(stream))


def svdq_i8_quantize_act(X, lam, M, K, qa, sa, stream=None):
    _entries.call("svdq_i8_quantize_act", ptr(X), ptr(lam), M, K, ptr(qa), ptr(sa),
                  stream_ptr(stream))


def svdq_i8_gemm_workspace_bytes(M, N, K) -> int:
    return int(_entries["svdq_i8_gemm_workspace_bytes"](M, N, K))


def svdq_i8_gemm(qa, sa, qw, sw, bias, act, M, N, K, Y, workspace, ws_bytes, stream=None):
    _entries.call("svdq_i8_gemm", ptr(qa), ptr(sa), ptr(qw), ptr(sw), ptr(bias), act, M, N, K,
                  ptr(Y), ptr(workspace), ws_bytes, stream_ptr(stream))


def svdq_i8_linear_workspace_bytes(M, N, K) -> int:
    return int(_entries["svdq_i8_linear_workspace_bytes"](M, N, K))


def svdq_i8_linear(X, lam, qw, sw, bias, act, M, N, K, Y, workspace, ws_bytes, stream=None):
    _entries.call("svdq_i8_linear", ptr(X), ptr(lam), ptr(qw), ptr(sw), ptr(bias), act, M, N, K,
                  ptr(Y), ptr(workspace), ws_bytes, stream_ptr(stream))


# ------------------------------------------------------------- tensor level

def i8_pack_weights(W: torch.Tensor):
    """fp32 weight [N, K] -> (qw int8 [N, K], sw fp32 [N])."""
    N, K = expect(W, "W", F32, (None, None))
    dev = one_device(W=W)
    qw = torch.empty((N, K), dtype=torch.int8, device=dev)
    sw = torch.empty(N, dtype=torch.float32, device=dev)
    with on(dev):
        _entries.call("svdq_i8_pack_weights", at(W), N, K, at(qw), at(sw), stream_ptr())
    return qw, sw


def i8_quantize_act(X: torch.Tensor, lam: Optional[torch.Tensor] = None):
    """X bf16 [M, K], smoothed by 1 / lam fp32 [K] if given -> (qa int8 [M, K], sa fp32 [M])."""
    M, K = expect(X, "X", BF16, (None, None))
    if lam is not None:
        expect(lam, "lam", F32, (K,))
    dev = one_device(X=X, lam=lam)
    qa = torch.empty((M, K), dtype=torch.int8, device=dev)
    sa = torch.empty(M, dtype=torch.float32, device=dev)
    with on(dev):
        _entries.call("svdq_i8_quantize_act", at(X), at(lam), M, K, at(qa), at(sa), stream_ptr())
    return qa, sa


def _weight(qw, sw, bias, K):
    N = expect(qw, "qw", I8, (None, K))[0]
    expect(sw, "sw", F32, (N,))
    if bias is not None:
        expect(bias, "bias", BF16, (N,))
    return N


def i8_gemm(qa, sa, qw, sw, bias=None, act: int = ACT_NONE,
            workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """act((qa qw^T) sa sw + bias) -> Y bf16 [M, N]; codes in [-127, 127]."""
    M, K = expect(qa, "qa", I8, (None, None))
    expect(sa, "sa", F32, (M,))
    N = _weight(qw, sw, bias, K)
    dev = one_device(qa=qa, sa=sa, qw=qw, sw=sw, bias=bias)
    need = svdq_i8_gemm_workspace_bytes(M, N, K)
    ws = scratch(workspace, need, dev)
    Y = qa.new_empty((M, N), dtype=torch.bfloat16)
    with on(dev):
        _entries.call("svdq_i8_gemm", at(qa), at(sa), at(qw), at(sw), at(bias), act, M, N, K, at(Y),
                      at(ws), need, stream_ptr())
    return Y


def i8_linear(X, lam, qw, sw, bias=None, act: int = ACT_NONE,
              workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The whole 8-bit layer: X bf16 [M, K] -> Y bf16 [M, N] (lam fp32 [K] or None; qw, sw from
    i8_pack_weights, or int8 codes in [-127, 127] and channel scales made elsewhere)."""
    M, K = expect(X, "X", BF16, (None, None))
    if lam is not None:
        expect(lam, "lam", F32, (K,))
    N = _weight(qw, sw, bias, K)
    dev = one_device(X=X, lam=lam, qw=qw, sw=sw, bias=bias)
    need = svdq_i8_linear_workspace_bytes(M, N, K)
    ws = scratch(workspace, need, dev)
    Y = X.new_empty((M, N), dtype=torch.bfloat16)
    with on(dev):
        _entries.call("svdq_i8_linear", at(X), at(lam), at(qw), at(sw), at(bias), act, M, N, K,
                      at(Y), at(ws), need, stream_ptr())
    return Y


class I8Linear:
    """An 8-bit replacement for one linear layer, beside SVDQLinear for the layers that lose
    too much in 4 bits: ``from_weight`` packs the weight (times the smoothing factors that the
    activations are divided by) on the GPU once, ``__call__`` runs the layer."""

    def __init__(self, lam, qw, sw, bias=None, act: int = ACT_NONE):
        self.lam, self.qw, self.sw, self.bias, self.act = lam, qw, sw, bias, act

    @classmethod
    def from_weight(cls, W, lam=None, bias=None, act: int = ACT_NONE):
        """W fp32 [N, K] of Y = X W^T; lam fp32 [K] smooths the activations (X / lam, W lam)."""
        qw, sw = i8_pack_weights(W if lam is None else W * lam)
        return cls(lam, qw, sw, bias, act)

    @property
    def in_features(self) -> int:
        return self.qw.shape[1]

    @property
    def out_features(self) -> int:
        return self.qw.shape[0]

    def __call__(self, X: torch.Tensor) -> torch.Tensor:
        return i8_linear(X, self.lam, self.qw, self.sw, self.bias, self.act)

"""The C ABI of include/svdq_i8.h: exports, refusals before any device call, and the tensor
checks.  The fake pointers are never dereferenced."""
import ctypes
import os
import re

import pytest
import torch

import bit_diffusion_transformer_amd as bdt
from bit_diffusion_transformer_amd import _binding, _int8

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include",
                      "svdq_i8.h")
OK, INVALID, SHAPE, MISALIGNED, WS_SMALL, NODEV, HIPERR = range(7)
A, U = 0x10000, 0x10008
P = ctypes.c_void_p
fn = _int8._entries


def last():
    return _binding.load_library().svdq_last_error()


def test_every_declared_symbol_is_exported():
    decl = sorted(set(re.findall(r"^[a-z_0-9 ]+\**\s*\**(svdq_\w+)\(", open(HEADER).read(), re.M)))
    assert decl == sorted(bdt.EXPORTS_I8)
    for name in decl:
        assert fn[name] is not None


def _pack(W=A, N=16, K=128, qw=A, sw=A):
    return fn["svdq_i8_pack_weights"](P(W), N, K, P(qw), P(sw), None)


def _quant(X=A, lam=A, M=16, K=128, qa=A, sa=A):
    return fn["svdq_i8_quantize_act"](P(X), P(lam), M, K, P(qa), P(sa), None)


def _gemm(qa=A, sa=A, qw=A, sw=A, bias=A, act=0, M=16, N=64, K=128, Y=A, ws=A, ws_bytes=1 << 40):
    return fn["svdq_i8_gemm"](P(qa), P(sa), P(qw), P(sw), P(bias), act, M, N, K, P(Y), P(ws),
                              ws_bytes, None)


def _lin(X=A, lam=A, qw=A, sw=A, bias=A, act=0, M=16, N=64, K=128, Y=A, ws=A, ws_bytes=1 << 40):
    return fn["svdq_i8_linear"](P(X), P(lam), P(qw), P(sw), P(bias), act, M, N, K, P(Y), P(ws),
                                ws_bytes, None)


BIG_K = (1 << 17) + 64


@pytest.mark.parametrize("call,kw,code", [
    (_pack, dict(N=-1), INVALID), (_pack, dict(N=(1 << 28) + 1), SHAPE), (_pack, dict(K=32), SHAPE),
    (_pack, dict(K=100), SHAPE), (_pack, dict(K=BIG_K), SHAPE), (_pack, dict(W=0), INVALID),
    (_pack, dict(qw=U), MISALIGNED), (_pack, dict(sw=0), INVALID),
    (_quant, dict(M=-1), INVALID), (_quant, dict(K=0), SHAPE), (_quant, dict(K=BIG_K), SHAPE),
    (_quant, dict(X=0), INVALID), (_quant, dict(lam=U), MISALIGNED), (_quant, dict(qa=U), MISALIGNED),
    (_quant, dict(sa=0), INVALID), (_quant, dict(M=(1 << 28)), SHAPE),
    (_gemm, dict(M=-1), INVALID), (_gemm, dict(act=2), INVALID), (_gemm, dict(N=12), SHAPE),
    (_gemm, dict(N=0), SHAPE), (_gemm, dict(K=96), SHAPE), (_gemm, dict(K=BIG_K), SHAPE),
    (_gemm, dict(qa=0), INVALID), (_gemm, dict(sa=U), MISALIGNED), (_gemm, dict(qw=0), INVALID),
    (_gemm, dict(sw=U), MISALIGNED), (_gemm, dict(bias=U), MISALIGNED), (_gemm, dict(Y=0), INVALID),
    (_gemm, dict(M=1 << 24, N=1 << 26), SHAPE),
    (_lin, dict(M=-1), INVALID), (_lin, dict(act=-1), INVALID), (_lin, dict(N=60), SHAPE),
    (_lin, dict(K=65), SHAPE), (_lin, dict(X=0), INVALID), (_lin, dict(lam=U), MISALIGNED),
    (_lin, dict(qw=U), MISALIGNED), (_lin, dict(sw=0), INVALID), (_lin, dict(Y=U), MISALIGNED),
    (_lin, dict(bias=U), MISALIGNED), (_lin, dict(ws_bytes=100), WS_SMALL), (_lin, dict(ws=0), INVALID),
    (_lin, dict(ws=U), MISALIGNED),
])
def test_rejects(call, kw, code):
    assert call(**kw) == code
    assert last()


def test_empty_inputs_are_noops():
    assert _pack(W=0, N=0, qw=0, sw=0) == OK
    assert _quant(X=0, lam=0, M=0, qa=0, sa=0) == OK
    assert _gemm(qa=0, sa=0, qw=0, sw=0, bias=0, M=0, Y=0, ws=0, ws_bytes=0) == OK
    assert _lin(X=0, lam=0, qw=0, sw=0, bias=0, M=0, Y=0, ws=0, ws_bytes=0) == OK
    if not torch.cuda.is_available():   # valid arguments: lambda and bias may be NULL
        assert _lin(lam=0, bias=0) == NODEV


def test_workspace_sizes():
    assert bdt.svdq_i8_linear_workspace_bytes(-1, 64, 128) == 0
    assert bdt.svdq_i8_gemm_workspace_bytes(1, -8, 128) == 0
    lin = bdt.svdq_i8_linear_workspace_bytes(100, 64, 192)
    assert lin == 19200 + 512 + bdt.svdq_i8_gemm_workspace_bytes(100, 64, 192)


def test_tensor_functions_refuse_bad_tensors():
    X, qw = torch.zeros(3, 128, dtype=torch.bfloat16), torch.zeros(16, 128, dtype=torch.int8)
    sw = torch.zeros(16)
    with pytest.raises(ValueError, match="GPU"):
        bdt.i8_linear(X, None, qw, sw)
    with pytest.raises(ValueError, match="shape"):
        bdt.i8_linear(X, None, qw[:, :64].contiguous(), sw)
    with pytest.raises(ValueError, match="shape"):
        bdt.i8_linear(X, torch.ones(64), qw, sw)
    with pytest.raises(ValueError, match="shape"):
        bdt.i8_linear(X, None, qw, sw[:8])
    with pytest.raises(TypeError):
        bdt.i8_linear(X.float(), None, qw, sw)
    with pytest.raises(TypeError):
        bdt.i8_linear(X, None, qw.to(torch.uint8), sw)
    with pytest.raises(TypeError):
        bdt.i8_linear(X, None, qw, sw, bias=sw)
    with pytest.raises(ValueError, match="contiguous"):
        bdt.i8_linear(X, None, torch.zeros(128, 16, dtype=torch.int8).t(), sw)
    with pytest.raises(ValueError, match="GPU"):
        bdt.i8_pack_weights(torch.zeros(16, 128))
    with pytest.raises(ValueError, match="GPU"):
        bdt.i8_quantize_act(X)
    with pytest.raises(ValueError, match="shape"):
        bdt.i8_gemm(qw, torch.zeros(3), qw, sw)

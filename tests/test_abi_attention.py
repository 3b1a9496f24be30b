"""The C ABI of include/svdq_attention.h: every declared symbol is exported and bad arguments
are refused before a device is touched; the tensor-level functions refuse bad tensors.

The fake pointers are never dereferenced: every call fails argument validation, which runs
before the device check and before any launch.
"""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import bit_diffusion_transformer_amd as bdt
from bit_diffusion_transformer_amd import _attention, _binding

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "svdq_attention.h")
OK, INVALID, SHAPE, MISALIGNED, WS_SMALL, NODEV, HIPERR = range(7)
A, U = 0x10000, 0x10008
P = ctypes.c_void_p


def declared_functions():
    return sorted(set(re.findall(r"^[a-z_0-9 ]+\**\s*\**(svdq_\w+)\(", open(HEADER).read(), re.M)))


@pytest.fixture(scope="module")
def fn():
    return _attention._entries


def last():
    return _binding.load_library().svdq_last_error()


def test_every_declared_symbol_is_exported(fn):
    decl = declared_functions()
    assert decl == sorted(bdt.EXPORTS_ATTENTION)
    for name in decl:
        assert fn[name] is not None


def _layout(tmp_path, struct, cls):
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "svdq_attention.h"\n'
                   'int main(void) { printf("%%zu", sizeof(%s));\n' % struct
                   + "".join('printf(" %%zu", offsetof(%s, %s));\n' % (struct, f)
                             for f, _ in cls._fields_) + "return 0; }\n")
    exe = tmp_path / "layout"
    subprocess.check_call(["gcc", "-I", os.path.dirname(HEADER), str(src), "-o", str(exe)])
    got = [int(v) for v in subprocess.check_output([str(exe)]).split()]
    assert got == [ctypes.sizeof(cls)] + [getattr(cls, f).offset for f, _ in cls._fields_]


def test_rope_axes_layout_matches_header(tmp_path):
    _layout(tmp_path, "svdq_rope_axes", bdt.RopeAxes)


def _tables(fn, pos=A, S=8, axes=None, cos=A, sin=A):
    axes = bdt.rope_axes((16, 56, 56)) if axes is None else axes
    return fn["svdq_rope_tables"](P(pos), S, axes and ctypes.byref(axes), P(cos), P(sin), None)


def _axes(n, dims, theta=10000.0):
    a = bdt.RopeAxes(axes=n)
    for i, d in enumerate(dims):
        a.dims[i], a.theta[i] = d, theta
    return a


@pytest.mark.parametrize("kw,code", [
    (dict(S=-1), INVALID), (dict(S=(1 << 28) + 1), SHAPE),
    (dict(axes=_axes(0, [])), INVALID), (dict(axes=_axes(5, [16] * 4)), INVALID),
    (dict(axes=_axes(2, [15, 17])), SHAPE), (dict(axes=_axes(2, [0, 16])), SHAPE),
    (dict(axes=_axes(2, [16, -16])), SHAPE), (dict(axes=_axes(1, [20])), SHAPE),
    (dict(axes=_axes(2, [128, 136])), SHAPE), (dict(axes=_axes(1, [64], 0.0)), INVALID),
    (dict(axes=_axes(1, [64], float("inf"))), INVALID),
    (dict(axes=_axes(1, [64], float("nan"))), INVALID),
    (dict(pos=0), INVALID), (dict(cos=0), INVALID), (dict(sin=0), INVALID),
    (dict(pos=U), MISALIGNED), (dict(sin=U), MISALIGNED),
])
def test_rope_tables_rejects(fn, kw, code):
    assert _tables(fn, **kw) == code
    assert last()


def test_rope_tables_rejects_null_axes_and_empty_is_a_noop(fn):
    assert fn["svdq_rope_tables"](P(A), 8, None, P(A), P(A), None) == INVALID
    assert _tables(fn, S=0, pos=0, cos=0, sin=0) == OK


def _epi(**kw):
    e = dict(heads=2, head_dim=128, seq=4, gamma_q=A, gamma_k=A, eps=1e-6, cos_t=A, sin_t=A,
             q=A, k=A, v=A)
    e.update(kw)
    return _binding.QkvEpilogue(**e)


@pytest.mark.parametrize("M,kw,code", [
    (-1, {}, INVALID), ((1 << 28) + 4, {}, SHAPE), (8, dict(head_dim=96), SHAPE),
    (8, dict(heads=1, head_dim=64), SHAPE), (8, dict(heads=0), INVALID), (8, dict(seq=3), SHAPE),
    (8, dict(seq=0), INVALID), (8, dict(eps=-1.0), INVALID), (8, dict(eps=float("nan")), INVALID),
    (8, dict(gamma_q=U), MISALIGNED), (8, dict(cos_t=None), INVALID), (8, dict(sin_t=U), MISALIGNED),
    (8, dict(q=None), INVALID), (8, dict(v=U), MISALIGNED), (8, dict(heads=1 << 21), SHAPE),
    (1 << 28, dict(heads=8192), SHAPE),
])
def test_qkv_norm_rope_rejects(fn, M, kw, code):
    assert fn["svdq_qkv_norm_rope"](P(A), M, ctypes.byref(_epi(**kw)), None) == code
    assert last()


def test_qkv_norm_rope_rejects_pointers_and_empty_is_a_noop(fn):
    call = fn["svdq_qkv_norm_rope"]
    assert call(P(A), 8, None, None) == INVALID
    assert call(P(0), 8, ctypes.byref(_epi()), None) == INVALID
    assert call(P(U), 8, ctypes.byref(_epi()), None) == MISALIGNED
    none = dict(q=None, k=None, v=None, gamma_q=None, gamma_k=None, cos_t=None, sin_t=None)
    assert call(P(0), 0, ctypes.byref(_epi(**none)), None) == OK
    if not torch.cuda.is_available():   # valid arguments, gamma NULL allowed: the device check
        assert call(P(A), 8, ctypes.byref(_epi(gamma_q=None, gamma_k=None)), None) == NODEV


def test_tensor_functions_refuse_bad_tensors():
    pos = torch.zeros(4, 3)
    with pytest.raises(ValueError, match="GPU"):
        bdt.rope_tables(pos, (16, 56, 56))
    with pytest.raises(ValueError, match="shape"):
        bdt.rope_tables(pos, (64, 64))
    with pytest.raises(TypeError):
        bdt.rope_tables(pos.double(), (16, 56, 56))
    with pytest.raises(ValueError, match="contiguous"):
        bdt.rope_tables(torch.zeros(3, 4).t(), (16, 56, 56))
    with pytest.raises(ValueError):
        bdt.rope_tables(pos, (16, 56, 56), theta=(1e4, 1e4))
    with pytest.raises(ValueError):
        bdt.rope_tables(torch.zeros(4, 5), (16,) * 5)
    with pytest.raises(ValueError, match="range"):
        bdt.rope_axes((2 ** 32 + 16,))
    with pytest.raises(ValueError, match="range"):
        bdt.select_blocks(torch.zeros(1, 1, 1, 64, dtype=torch.bfloat16),
                          torch.zeros(1, 1, 1, 64, dtype=torch.bfloat16), 2 ** 32 + 1)
    qkv = torch.zeros(8, 3 * 2 * 64, dtype=torch.bfloat16)
    t = torch.zeros(4, 32)
    with pytest.raises(ValueError, match="GPU"):
        bdt.qkv_norm_rope(qkv, 2, 64, 4, None, None, 1e-6, t, t)
    with pytest.raises(ValueError, match="shape"):
        bdt.qkv_norm_rope(qkv, 2, 128, 4, None, None, 1e-6, t, t)
    with pytest.raises(ValueError, match="shape"):
        bdt.qkv_norm_rope(qkv, 2, 64, 5, None, None, 1e-6, t, t)
    with pytest.raises(ValueError, match="multiple"):
        bdt.qkv_norm_rope(qkv[:7], 2, 64, 4, None, None, 1e-6, t, t)
    with pytest.raises(TypeError):
        bdt.qkv_norm_rope(qkv.float(), 2, 64, 4, None, None, 1e-6, t, t)


# ---------------------------------------------------------------- sparse attention

def test_attention_shape_layout_matches_header(tmp_path):
    _layout(tmp_path, "svdq_attention_shape", bdt.AttentionShape)


def _shape(**kw):
    s = dict(batch=2, seq_q=200, seq_k=300, heads=4, kv_heads=2, head_dim=128, keep=3, first=1)
    s.update(kw)
    return bdt.AttentionShape(**s)


def _select(fn, shape=None, q=A, k=A, kv_len=0, blocks=A, ws=A, ws_bytes=1 << 40):
    return fn["svdq_select_blocks"](P(q), P(k), P(kv_len), ctypes.byref(shape or _shape()),
                                    P(blocks), P(ws), ws_bytes, None)


def _block(fn, shape=None, q=A, k=A, v=A, kv_len=0, scale=0.1, blocks=A, out=A, ws=A,
           ws_bytes=1 << 40):
    return fn["svdq_block_attention"](P(q), P(k), P(v), P(kv_len), ctypes.byref(shape or _shape()),
                                      scale, P(blocks), P(out), P(ws), ws_bytes, None)


def _sparse(fn, shape=None, q=A, k=A, v=A, kv_len=0, scale=0.1, blocks=0, out=A, ws=A,
            ws_bytes=1 << 40):
    return fn["svdq_sparse_attention"](P(q), P(k), P(v), P(kv_len), ctypes.byref(shape or _shape()),
                                       scale, P(blocks), P(out), P(ws), ws_bytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(batch=-1), INVALID), (dict(seq_q=-1), INVALID), (dict(batch=(1 << 28) + 1), SHAPE),
    (dict(seq_k=0), SHAPE), (dict(seq_k=-5), SHAPE), (dict(seq_k=(1 << 18) + 1), SHAPE),
    (dict(heads=0), INVALID), (dict(heads=-4), INVALID), (dict(kv_heads=0), SHAPE),
    (dict(kv_heads=3), SHAPE), (dict(kv_heads=-2), SHAPE), (dict(head_dim=96), SHAPE),
    (dict(head_dim=256), SHAPE), (dict(keep=0), SHAPE), (dict(keep=4097), SHAPE),
    (dict(first=-1), INVALID), (dict(first=4), INVALID),
    (dict(batch=1 << 27, heads=4), SHAPE), (dict(batch=1 << 10, heads=1 << 10, seq_q=1 << 20), SHAPE),
    (dict(batch=1 << 20, seq_k=1 << 18), SHAPE),
])
def test_sparse_attention_rejects_shapes(fn, kw, code):
    for call in (_select, _block, _sparse):
        assert call(fn, _shape(**kw)) == code
        assert last()
    for size in ("select_blocks", "block_attention", "sparse_attention"):
        assert fn["svdq_%s_workspace_bytes" % size](ctypes.byref(_shape(**kw))) == 0


@pytest.mark.parametrize("call,kw,code", [
    (_select, dict(q=0), INVALID), (_select, dict(k=U), MISALIGNED), (_select, dict(kv_len=U), MISALIGNED),
    (_select, dict(blocks=0), INVALID), (_select, dict(ws=0), INVALID), (_select, dict(ws_bytes=8), WS_SMALL),
    (_block, dict(q=U), MISALIGNED), (_block, dict(k=0), INVALID), (_block, dict(v=0), INVALID),
    (_block, dict(blocks=U), MISALIGNED), (_block, dict(out=0), INVALID), (_block, dict(kv_len=U), MISALIGNED),
    (_block, dict(scale=0.0), INVALID), (_block, dict(scale=-1.0), INVALID),
    (_block, dict(scale=float("inf")), INVALID), (_block, dict(scale=float("nan")), INVALID),
    (_sparse, dict(q=0), INVALID), (_sparse, dict(v=U), MISALIGNED), (_sparse, dict(out=U), MISALIGNED),
    (_sparse, dict(blocks=U), MISALIGNED), (_sparse, dict(scale=float("nan")), INVALID),
    (_sparse, dict(ws=U), MISALIGNED), (_sparse, dict(ws_bytes=8), WS_SMALL),
])
def test_sparse_attention_rejects_arguments(fn, call, kw, code):
    assert call(fn, **kw) == code
    assert last()


def test_sparse_attention_null_shape_and_empty(fn):
    assert fn["svdq_select_blocks"](P(A), P(A), None, None, P(A), P(A), 1 << 40, None) == INVALID
    for kw in (dict(batch=0), dict(seq_q=0)):
        s = _shape(**kw)
        assert _select(fn, s, q=0, k=0, blocks=0, ws=0, ws_bytes=0) == OK
        assert _block(fn, s, q=0, k=0, v=0, blocks=0, out=0, ws=0, ws_bytes=0) == OK
        assert _sparse(fn, s, q=0, k=0, v=0, out=0, ws=0, ws_bytes=0) == OK
        assert bdt.svdq_sparse_attention_workspace_bytes(s) == 0


def test_sparse_attention_workspace_sizes():
    # 64-bit means of 2 x 4 x 2 query and 2 x 2 x 5 key blocks of 128 columns, in tiles of 16
    means = 2 * 4 * 16 * 128 * 8 + 2 * 2 * 16 * 128 * 8
    assert bdt.svdq_select_blocks_workspace_bytes(_shape()) == means
    assert bdt.svdq_sparse_attention_workspace_bytes(_shape()) >= means + 2 * 4 * 2 * 3 * 4
    assert bdt.svdq_block_attention_workspace_bytes(_shape(batch=64, seq_q=4096)) == 0


def test_attention_tensor_functions_refuse_bad_tensors():
    bf = torch.bfloat16
    q, k = torch.zeros(2, 4, 200, 64, dtype=bf), torch.zeros(2, 2, 300, 64, dtype=bf)
    blocks = torch.zeros(2, 4, 2, 3, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        bdt.sparse_attention(q, k, k, 3)
    with pytest.raises(ValueError, match="GPU"):
        bdt.select_blocks(q, k, 3)
    with pytest.raises(ValueError, match="GPU"):
        bdt.block_attention(q, k, k, blocks)
    with pytest.raises(ValueError, match="shape"):
        bdt.block_attention(q, k, k, blocks[:, :, :1].contiguous())
    with pytest.raises(ValueError, match="shape"):
        bdt.sparse_attention(q, k, k[:, :, :299].contiguous(), 3)
    with pytest.raises(ValueError, match="shape"):
        bdt.sparse_attention(q, k[..., :32].contiguous(), k, 3)
    with pytest.raises(ValueError, match="contiguous"):
        bdt.sparse_attention(q.transpose(1, 2).contiguous().transpose(1, 2), k, k, 3)
    with pytest.raises(TypeError):
        bdt.sparse_attention(q.float(), k, k, 3)
    with pytest.raises(TypeError):
        bdt.sparse_attention(q, k, k, 3, kv_len=torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="shape"):
        bdt.sparse_attention(q, k, k, 3, kv_len=torch.zeros(3, dtype=torch.int32))

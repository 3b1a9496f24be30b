"""The C ABI of include/svdq_paged.h: every declared symbol is exported and bad arguments are
refused before a device is touched; the tensor-level functions refuse bad tensors.

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
from bit_diffusion_transformer_amd import _binding, _paged

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "svdq_paged.h")
OK, INVALID, SHAPE, MISALIGNED, WS_SMALL, NODEV, HIPERR = range(7)
A, U, I = 0x10000, 0x10008, 0x10002   # I: of an int32 array
P = ctypes.c_void_p
BF, I32 = torch.bfloat16, torch.int32


@pytest.fixture(scope="module")
def fn():
    return _paged._entries


def last():
    return _binding.load_library().svdq_last_error()


def test_every_declared_symbol_is_exported(fn):
    decl = sorted(set(re.findall(r"^[a-z_0-9 ]+\**\s*\**(svdq_\w+)\(", open(HEADER).read(), re.M)))
    assert decl == sorted(bdt.EXPORTS_PAGED)
    for name in decl:
        assert fn[name] is not None


@pytest.mark.parametrize("struct,cls", [
    ("svdq_packed_shape", bdt.PackedShape), ("svdq_paged_shape", bdt.PagedShape),
    ("svdq_table_shape", bdt.TableShape), ("svdq_cache_epilogue", bdt.CacheEpilogue)])
def test_struct_layouts_match_header(tmp_path, struct, cls):
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "svdq_paged.h"\n'
                   'int main(void) { printf("%%zu", sizeof(%s));\n' % struct
                   + "".join('printf(" %%zu", offsetof(%s, %s));\n' % (struct, f)
                             for f, _ in cls._fields_) + "return 0; }\n")
    exe = tmp_path / "layout"
    subprocess.check_call(["gcc", "-I", os.path.dirname(HEADER), str(src), "-o", str(exe)])
    got = [int(v) for v in subprocess.check_output([str(exe)]).split()]
    assert got == [ctypes.sizeof(cls)] + [getattr(cls, f).offset for f, _ in cls._fields_]


def packed(**kw):
    s = dict(tokens_q=100, tokens_k=100, q_stride=512, k_stride=256, v_stride=256, sequences=3, heads=4,
             kv_heads=2, head_dim=128, causal=1)
    s.update(kw)
    return bdt.PackedShape(**s)


def call_packed(fn, shape=None, q=A, k=A, v=A, at=A, kat=0, scale=0.1, out=A, ws=A, n=1 << 40):
    shape = packed() if shape is None else shape
    return fn["svdq_packed_attention"](P(q), P(k), P(v), P(at), P(kat), shape and ctypes.byref(shape),
                                       scale, P(out), P(ws), n, None)


HEADS = [(dict(heads=0), INVALID), (dict(kv_heads=0), SHAPE), (dict(kv_heads=3), SHAPE),
         (dict(heads=130, q_stride=130 * 128), SHAPE), (dict(head_dim=96), SHAPE), (dict(head_dim=256), SHAPE),
         (dict(causal=2), INVALID), (dict(causal=-1), INVALID), (dict(heads=1 << 22, kv_heads=1 << 20), SHAPE)]
STRIDES = [(dict(q_stride=504), SHAPE), (dict(q_stride=516), SHAPE), (dict(q_stride=(1 << 20) + 8), SHAPE),
           (dict(q_stride=-512), SHAPE)]


@pytest.mark.parametrize("kw,code", HEADS + STRIDES + [
    (dict(tokens_q=-1), INVALID), (dict(tokens_k=-1), INVALID), (dict(sequences=-1), INVALID),
    (dict(tokens_q=(1 << 28) + 1), SHAPE), (dict(sequences=(1 << 28) + 1), SHAPE),
    (dict(k_stride=248), SHAPE), (dict(v_stride=252), SHAPE), (dict(v_stride=0), SHAPE),
    (dict(tokens_k=99), INVALID),
    (dict(tokens_q=1 << 28, tokens_k=1 << 28, sequences=1 << 20), SHAPE)])
def test_packed_attention_rejects_shapes(fn, kw, code):
    assert call_packed(fn, packed(**kw)) == code
    assert last()
    if kw != dict(tokens_k=99):                      # (its own k_starts would allow that)
        assert fn["svdq_packed_attention_workspace_bytes"](ctypes.byref(packed(**kw))) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(q=0), INVALID), (dict(k=0), INVALID), (dict(v=0), INVALID), (dict(at=0), INVALID),
    (dict(out=0), INVALID), (dict(ws=0), INVALID), (dict(q=U), MISALIGNED), (dict(k=U), MISALIGNED),
    (dict(v=U), MISALIGNED), (dict(at=I), MISALIGNED), (dict(kat=I), MISALIGNED), (dict(out=U), MISALIGNED),
    (dict(ws=U), MISALIGNED), (dict(n=16), WS_SMALL), (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID), (dict(scale=2.0 ** 127.5), INVALID)])
def test_packed_attention_rejects_arguments(fn, kw, code):
    assert call_packed(fn, **kw) == code
    assert last()


def test_packed_attention_null_shape_and_empty(fn):
    assert fn["svdq_packed_attention"](P(A), P(A), P(A), P(A), P(0), None, 0.1, P(A), P(A), 1 << 30, None) == INVALID
    assert fn["svdq_packed_attention_workspace_bytes"](None) == 0
    for kw in (dict(tokens_q=0, tokens_k=0), dict(sequences=0)):
        assert call_packed(fn, packed(**kw), 0, 0, 0, 0, 0, 0.1, 0, 0, 0) == OK
        assert fn["svdq_packed_attention_workspace_bytes"](ctypes.byref(packed(**kw))) == 0
    if not torch.cuda.is_available():
        assert call_packed(fn) == NODEV
        assert call_packed(fn, packed(tokens_k=7), kat=A) == NODEV
        assert call_packed(fn, packed(tokens_k=0), k=0, v=0, kat=A) == NODEV


def paged(**kw):
    s = dict(tokens=10, pages=50, q_stride=512, requests=3, heads=4, kv_heads=2, head_dim=128, page=16, width=9,
             max_new=4, causal=1)
    s.update(kw)
    return bdt.PagedShape(**s)


def call_paged(fn, shape=None, q=A, k=A, v=A, t=A, at=A, kv=A, scale=0.1, out=A, ws=A, n=1 << 40):
    shape = paged() if shape is None else shape
    return fn["svdq_paged_attention"](P(q), P(k), P(v), P(t), P(at), P(kv), shape and ctypes.byref(shape), scale,
                                      P(out), P(ws), n, None)


PAGES = [(dict(page=0), SHAPE), (dict(page=8), SHAPE), (dict(page=24), SHAPE), (dict(page=512), SHAPE),
         (dict(page=-16), SHAPE), (dict(pages=-1), INVALID), (dict(pages=(1 << 26) + 1), SHAPE)]


@pytest.mark.parametrize("kw,code", HEADS + STRIDES + PAGES + [
    (dict(tokens=-1), INVALID), (dict(tokens=(1 << 28) + 1), SHAPE), (dict(requests=-1), INVALID),
    (dict(width=-1), INVALID), (dict(width=(1 << 26) + 1), SHAPE), (dict(max_new=0), INVALID),
    (dict(max_new=-3), INVALID)])
def test_paged_attention_rejects_shapes(fn, kw, code):
    assert call_paged(fn, paged(**kw)) == code
    assert last()
    assert fn["svdq_paged_attention_workspace_bytes"](ctypes.byref(paged(**kw))) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(q=0), INVALID), (dict(k=0), INVALID), (dict(v=0), INVALID), (dict(t=0), INVALID), (dict(at=0), INVALID),
    (dict(kv=0), INVALID), (dict(out=0), INVALID), (dict(ws=0), INVALID), (dict(q=U), MISALIGNED),
    (dict(k=U), MISALIGNED), (dict(v=U), MISALIGNED), (dict(t=I), MISALIGNED), (dict(at=I), MISALIGNED),
    (dict(kv=I), MISALIGNED), (dict(out=U), MISALIGNED), (dict(ws=U), MISALIGNED), (dict(n=16), WS_SMALL),
    (dict(scale=0.0), INVALID), (dict(scale=float("nan")), INVALID)])
def test_paged_attention_rejects_arguments(fn, kw, code):
    assert call_paged(fn, **kw) == code
    assert last()


def test_paged_attention_null_shape_and_empty(fn):
    assert fn["svdq_paged_attention"](P(A), P(A), P(A), P(A), P(A), P(A), None, 0.1, P(A), P(A), 1 << 30,
                                      None) == INVALID
    assert fn["svdq_paged_attention_workspace_bytes"](None) == 0
    for kw in (dict(tokens=0), dict(requests=0)):
        assert call_paged(fn, paged(**kw), 0, 0, 0, 0, 0, 0, 0.1, 0, 0, 0) == OK
    if not torch.cuda.is_available():
        assert call_paged(fn) == NODEV
        assert call_paged(fn, paged(pages=0), k=0, v=0) == NODEV
        assert call_paged(fn, paged(width=0), t=0) == NODEV


@pytest.mark.parametrize("D", [64, 128])
def test_workspace_grows_to_a_limit(fn, D):
    """Not with the keys or requests past what the workgroups at once need."""
    def need(**kw):
        return fn["svdq_paged_attention_workspace_bytes"](ctypes.byref(paged(head_dim=D, q_stride=64 * D, **kw)))
    small = need(tokens=1, requests=1, width=1, heads=1, kv_heads=1)
    most = need(tokens=4000, requests=4000, width=1 << 16, heads=64, kv_heads=8)
    assert 0 < small < most < 200 << 20
    assert need(tokens=1 << 20, requests=1 << 10, width=1 << 20, heads=64, kv_heads=64, max_new=1 << 10) < 200 << 20


def call_tables(fn, shape, cached=A, added=A, free=A, tables=A, at=A, kv=A, slots=A, pos=A, counts=A):
    return fn["svdq_page_tables"](P(cached), P(added), P(free), shape and ctypes.byref(shape), P(tables), P(at), P(kv),
                                  P(slots), P(pos), P(counts), None)


def table(**kw):
    s = dict(tokens=10, pages=50, free_count=20, requests=3, page=16, width=9)
    s.update(kw)
    return bdt.TableShape(**s)


@pytest.mark.parametrize("kw,code", PAGES + [
    (dict(tokens=-1), INVALID), (dict(tokens=(1 << 28) + 1), SHAPE), (dict(free_count=-1), INVALID),
    (dict(requests=-1), INVALID), (dict(requests=8193), SHAPE), (dict(width=-1), INVALID)])
def test_page_tables_rejects_shapes(fn, kw, code):
    assert call_tables(fn, table(**kw)) == code
    assert last()


@pytest.mark.parametrize("what", ["cached", "added", "free", "tables", "at", "kv", "slots", "pos", "counts"])
def test_page_tables_rejects_pointers(fn, what):
    assert call_tables(fn, table(), **{what: 0}) == INVALID
    assert call_tables(fn, table(), **{what: I}) == MISALIGNED
    assert call_tables(fn, None) == INVALID
    if not torch.cuda.is_available():
        assert call_tables(fn, table()) == NODEV
        assert call_tables(fn, table(requests=0, tokens=0, free_count=0), 0, 0, 0, 0, A, 0, 0, 0, A) == NODEV


def epilogue(**kw):
    e = dict(tokens=10, table_rows=100, pages=50, heads=4, kv_heads=2, head_dim=128, rotary=64, half=1, page=16,
             gamma_q=A, gamma_k=A, eps=1e-6, cos_t=A, sin_t=A, positions=A, slots=A, q=A, k_cache=A, v_cache=A)
    e.update(kw)
    return bdt.CacheEpilogue(**e)


@pytest.mark.parametrize("kw,code", [(k, c) for k, c in HEADS if "causal" not in k and "q_stride" not in k] + PAGES + [
    (dict(heads=130), SHAPE), (dict(tokens=-1), INVALID), (dict(tokens=(1 << 28) + 1), SHAPE),
    (dict(tokens=1 << 28, heads=1024, kv_heads=64), SHAPE), (dict(table_rows=0), INVALID),
    (dict(table_rows=(1 << 28) + 1), SHAPE), (dict(rotary=0), SHAPE), (dict(rotary=8), SHAPE), (dict(rotary=40), SHAPE),
    (dict(rotary=144), SHAPE), (dict(half=2), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(eps=float("inf")), INVALID)]
    + [(dict([(n, None)]), INVALID) for n in ("cos_t", "sin_t", "positions", "slots", "q", "k_cache", "v_cache")]
    + [(dict([(n, U)]), MISALIGNED) for n in ("gamma_q", "gamma_k", "cos_t", "sin_t", "q", "k_cache", "v_cache")]
    + [(dict([(n, I)]), MISALIGNED) for n in ("positions", "slots")])
def test_cache_epilogue_rejects(fn, kw, code):
    assert fn["svdq_qkv_norm_rope_cache"](P(A), ctypes.byref(epilogue(**kw)), None) == code
    assert last()


def test_cache_epilogue_null_and_empty(fn):
    call = fn["svdq_qkv_norm_rope_cache"]
    assert call(P(A), None, None) == INVALID
    assert call(P(0), ctypes.byref(epilogue()), None) == INVALID
    assert call(P(U), ctypes.byref(epilogue()), None) == MISALIGNED
    assert call(P(0), ctypes.byref(epilogue(tokens=0, q=None, cos_t=None, slots=None)), None) == OK
    if not torch.cuda.is_available():
        assert call(P(A), ctypes.byref(epilogue(gamma_q=None, gamma_k=None)), None) == NODEV
        assert call(P(A), ctypes.byref(epilogue(pages=0, k_cache=None, v_cache=None)), None) == NODEV


# ------------------------------------------------------------------ tensors (on the CPU: refused in the end)

def z(*shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype)


def test_packed_attention_refuses_bad_tensors():
    q, k, at = z(5, 4, 64), z(5, 2, 64), z(3, dtype=I32)
    bad = [((q.float(), k, k, at), TypeError), ((q, k.half(), k, at), TypeError), ((q, k, z(5, 2, 128), at), ValueError),
           ((q, z(5, 2, 128), k, at), ValueError), ((q, k, z(4, 2, 64), at), ValueError), ((q, k, k, at.long()), TypeError),
           ((q, k, k, at[:0]), ValueError), ((q, z(6, 2, 64), z(6, 2, 64), at), ValueError),
           ((z(5, 64, 4).transpose(1, 2), k, k, at), ValueError), ((z(10, 4, 64)[::2], z(5, 4, 64)[:, ::2], k, at), ValueError),
           ((z(5, 4, 128)[:, :, ::2], k, k, at), ValueError), ((z(4, 64), k, k, at), ValueError), ((None, k, k, at), TypeError),
           ((z(1, 4, 64).expand(5, 4, 64), k, k, at), ValueError)]
    for args, error in bad:
        with pytest.raises(error):
            bdt.packed_attention(*args)
    with pytest.raises(ValueError, match="shape"):
        bdt.packed_attention(q, k, k, at, z(4, dtype=I32))
    with pytest.raises(ValueError, match="shape"):
        bdt.packed_attention(q, k, k, at, out=z(5, 4, 128))
    with pytest.raises(TypeError):
        bdt.packed_attention(q, k, k, at, out=z(5, 4, 64, dtype=torch.float16))
    for good in (q, z(5, 8, 64)[:, :4], z(5, 12 * 64)[:, 64:320].view(5, 4, 64)):
        with pytest.raises(ValueError, match="GPU"):
            bdt.packed_attention(good, k, k, at)


def test_paged_attention_refuses_bad_tensors():
    ok = dict(q=z(5, 4, 64), k_cache=z(7, 2, 16, 64), v_cache=z(7, 2, 16, 64), tables=z(3, 9, dtype=I32),
              q_starts=z(4, dtype=I32), kv_len=z(3, dtype=I32))
    with pytest.raises(ValueError, match="GPU"):
        bdt.paged_attention(**ok)
    for kw, error in ((dict(q=z(5, 4, 128)), ValueError), (dict(k_cache=z(7, 2, 32, 64)), ValueError),
                      (dict(v_cache=z(7, 3, 16, 64)), ValueError), (dict(tables=z(2, 9, dtype=I32)), ValueError),
                      (dict(tables=z(3, 9, dtype=torch.int64)), TypeError), (dict(q_starts=z(3, dtype=I32)), ValueError),
                      (dict(kv_len=z(4, dtype=I32)), ValueError), (dict(max_new=0), ValueError),
                      (dict(tables=z(9, 3, dtype=I32).t()), ValueError), (dict(out=z(5, 2, 64)), ValueError),
                      (dict(k_cache=z(7, 16, 2, 64).transpose(1, 2)), ValueError), (dict(q=None), TypeError)):
        with pytest.raises(error):
            bdt.paged_attention(**{**ok, **kw})


def test_page_tables_refuses_bad_tensors():
    i3 = z(3, dtype=I32)
    with pytest.raises(ValueError, match="GPU"):
        bdt.page_tables(i3, i3, i3, z(3, 5, dtype=I32), 16, 50, 10)
    for args, error in (((i3.long(), i3, i3, z(3, 5, dtype=I32), 16, 50, 10), TypeError),
                        ((i3, z(4, dtype=I32), i3, z(3, 5, dtype=I32), 16, 50, 10), ValueError),
                        ((i3, i3, i3, z(2, 5, dtype=I32), 16, 50, 10), ValueError),
                        ((i3, i3, i3, z(3, 5, dtype=I32), 2 ** 32 + 16, 50, 10), ValueError),
                        ((i3, i3, i3, z(3, 5, dtype=I32), 16, 2 ** 40, 10), ValueError),
                        ((i3, i3, i3, z(3, 5, dtype=I32), 16, 50, -1), ValueError)):
        with pytest.raises(error):
            bdt.page_tables(*args)


def test_qkv_norm_rope_cache_refuses_bad_tensors():
    i5, t = z(5, dtype=I32), z(9, 16, dtype=torch.float32)
    ok = dict(qkv=z(5, 8 * 64), heads=4, kv_heads=2, gamma_q=z(64), gamma_k=None, eps=1e-6, cos_t=t, sin_t=t,
              positions=i5, slots=i5, k_cache=z(7, 2, 16, 64), v_cache=z(7, 2, 16, 64))
    with pytest.raises(ValueError, match="GPU"):
        bdt.qkv_norm_rope_cache(**ok)
    for kw, error in ((dict(heads=5), ValueError), (dict(kv_heads=3), ValueError), (dict(gamma_q=z(128)), ValueError),
                      (dict(gamma_k=z(64).float()), TypeError), (dict(sin_t=z(9, 8, dtype=torch.float32)), ValueError),
                      (dict(cos_t=t.double()), TypeError), (dict(positions=z(4, dtype=I32)), ValueError),
                      (dict(slots=i5.long()), TypeError), (dict(v_cache=z(7, 2, 32, 64)), ValueError),
                      (dict(out=z(5, 4, 128)), ValueError), (dict(qkv=z(8 * 64, 5).t()), ValueError)):
        with pytest.raises(error):
            bdt.qkv_norm_rope_cache(**{**ok, **kw})

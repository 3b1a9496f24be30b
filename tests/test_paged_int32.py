"""Sizes that a C int32 does not hold are refused by the tensor-level functions (ctypes would drop
their higher bits and the library would see others).  Tensors without elements have any size."""
import pytest
import torch

import bit_diffusion_transformer_amd as bdt
from tests.test_cached_attention_call import _args
from tests.test_abi_paged import BF, I32, z

BIG = 1 << 32


@pytest.mark.parametrize("q,k", [((0, BIG + 4, 64), (0, 2, 64)), ((5, 4, 64), (0, BIG + 2, 64)), ((0, 4, BIG + 64), (0, 2, BIG + 64))])
def test_packed_attention(q, k):
    with pytest.raises(ValueError, match="range"):
        bdt.packed_attention(z(*q), z(*k), z(*k), z(2, dtype=I32), z(2, dtype=I32))


@pytest.mark.parametrize("kw", [
    dict(q=z(0, BIG + 4, 64)), dict(k_cache=z(0, 2, BIG + 16, 64), v_cache=z(0, 2, BIG + 16, 64)),
    dict(k_cache=z(0, BIG + 2, 16, 64), v_cache=z(0, BIG + 2, 16, 64)),
    dict(tables=z(0, BIG + 9, dtype=I32), q_starts=z(1, dtype=I32), kv_len=z(0, dtype=I32))])
def test_paged_attention(kw):
    ok = dict(q=z(5, 4, 64), k_cache=z(7, 2, 16, 64), v_cache=z(7, 2, 16, 64), tables=z(3, 9, dtype=I32),
              q_starts=z(4, dtype=I32), kv_len=z(3, dtype=I32))
    with pytest.raises(ValueError, match="range"):
        bdt.paged_attention(**{**ok, **kw})


def test_page_tables():
    i0 = z(0, dtype=I32)
    with pytest.raises(ValueError, match="range"):
        bdt.page_tables(i0, i0, i0, z(0, BIG + 5, dtype=I32), 16, 50, 10)


@pytest.mark.parametrize("heads,G,D,page", [(BIG + 4, 2, 64, 16), (4, BIG + 2, 64, 16), (4, 2, BIG + 64, 16), (4, 2, 64, BIG + 16)])
def test_qkv_norm_rope_cache(heads, G, D, page):
    t, i0, cache = z(9, 16, dtype=torch.float32), z(0, dtype=I32), z(0, G, page, D)
    with pytest.raises(ValueError, match="range"):
        bdt.qkv_norm_rope_cache(z(0, (heads + 2 * G) * D), heads, G, None, None, 1e-6, t, t, i0, i0, cache, cache)


@pytest.mark.parametrize("kw", [{n: torch.zeros(0, 2, BIG + 16, 64, dtype=BF) for n in ("k_cache", "v_cache")},
                                dict(tables=z(0, BIG + 4, dtype=I32), q_starts=z(1, dtype=I32), kv_len=z(0, dtype=I32))])
def test_cached_attention(kw):
    with pytest.raises(ValueError, match="range"):
        bdt.cached_attention(**_args(**kw))

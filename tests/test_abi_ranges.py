"""Arguments at the edges of the documented ranges: refused or taken before any device call.
The fake pointers are never dereferenced: a call that is taken ends at the device check of a
host without a GPU."""
import ctypes

import pytest
import torch

import bit_diffusion_transformer_amd as bdt
from bit_diffusion_transformer_amd import _attention, _binding, _int8

OK, INVALID, SHAPE, MISALIGNED, WS_SMALL, NODEV, HIPERR = range(7)
A, P = 0x10000, ctypes.c_void_p
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="the taken calls would launch")


@no_gpu
@pytest.mark.parametrize("scale,code", [(2.0 ** 127, NODEV), (1.8e38, INVALID), (3e38, INVALID),
                                        (1e-45, NODEV)])
def test_scale_of_the_attention(scale, code):
    """scale log2 e has to be finite too: an infinite one would make every weight NaN."""
    fn, s = _attention._entries, bdt.AttentionShape(2, 200, 300, 4, 2, 128, 3, 1)
    for name in ("svdq_block_attention", "svdq_sparse_attention"):
        got = fn[name](P(A), P(A), P(A), P(0), ctypes.byref(s), scale, P(A), P(A), P(A), 1 << 40, None)
        assert got == code, name
        assert _binding.svdq_last_error()


def test_raw_calls_refuse_tensors_that_are_not_contiguous():
    """The pointer alone does not tell the strides: like the raw calls of svdq.h, these raise
    before they reach the library."""
    t = torch.zeros(8, 8).t()
    with pytest.raises(ValueError, match="contiguous"):
        bdt.svdq_i8_pack_weights(t, 8, 8, None, None)
    with pytest.raises(ValueError, match="contiguous"):
        bdt.svdq_i8_quantize_act(None, t, 8, 64, None, None)
    with pytest.raises(ValueError, match="contiguous"):
        bdt.svdq_i8_gemm(None, None, t, None, None, 0, 8, 8, 64, None, None, 0)
    with pytest.raises(ValueError, match="contiguous"):
        bdt.svdq_i8_linear(None, None, None, None, None, 0, 8, 8, 64, None, t, 0)
    with pytest.raises(ValueError, match="contiguous"):
        bdt.svdq_rope_tables(t, 8, bdt.rope_axes((64,)), None, None)
    with pytest.raises(ValueError, match="contiguous"):
        bdt.svdq_qkv_norm_rope(t, 8, _binding.QkvEpilogue())
    s = bdt.AttentionShape(1, 8, 8, 1, 1, 64, 1, 0)
    with pytest.raises(ValueError, match="contiguous"):
        bdt.svdq_select_blocks(None, t, None, s, None, None, 0)
    with pytest.raises(ValueError, match="contiguous"):
        bdt.svdq_block_attention(None, None, t, None, s, 1.0, None, None, None, 0)
    with pytest.raises(ValueError, match="contiguous"):
        bdt.svdq_sparse_attention(None, None, None, None, s, 1.0, None, t, None, 0)


@no_gpu
@pytest.mark.parametrize("rows,K,code", [
    (1 << 23, 64, NODEV), ((1 << 26) - 4, 4096, NODEV), ((1 << 26) + 4, 4096, SHAPE),
    ((1 << 25) - 4, 8192, NODEV), ((1 << 25) + 4, 8192, SHAPE),
    ((1 << 23) - 1, 16448, NODEV), (1 << 23, 16448, SHAPE)])
def test_rows_of_the_8bit_quantizer(rows, K, code):
    """As many as its launch takes: four a workgroup of 256 (512 from K = 4160 on), one of 512
    past K = 16384; 2^32 - 1 work-items."""
    fn = _int8._entries
    assert fn["svdq_i8_quantize_act"](P(A), P(0), rows, K, P(A), P(A), None) == code
    assert fn["svdq_i8_pack_weights"](P(A), rows, K, P(A), P(A), None) == code
    assert fn["svdq_i8_linear"](P(A), P(0), P(A), P(A), P(0), 0, rows, 8, K, P(A), P(A), 1 << 60, None) == code

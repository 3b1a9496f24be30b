"""The attentions of packed and paged sequences divide a line of tiles whose positions are whole
numbers, over a cache quarters, in 64-bit floating point: exact up to 2^53 of them.  Longer
lines are refused, and starts that descend cannot name one."""
import ctypes

import pytest
import torch

import bit_diffusion_transformer_amd as bdt
from bit_diffusion_transformer_amd import _paged
from tests.test_abi_paged import OK, SHAPE, call_packed, call_paged, packed, paged

BF = torch.bfloat16


def longest(T, Tk, B, H, G):
    """At least the line's length: T group / 16 + B tiles a key head, each at most (keys + rows +
    512) group + 256 (512: what a narrow tile costs beside its keys)."""
    g = H // G
    return (T * g / 16 + B) * (g * (Tk + T + 512) + 256) * G


@pytest.mark.parametrize("T,B,width,H,G", [(1 << 20, 1 << 10, 1 << 20, 64, 8), (1 << 24, 1 << 24, 1 << 12, 8, 8),
                                           (1 << 18, 1 << 18, 1 << 16, 128, 2), (1, 1 << 28, 1 << 14, 64, 64)])
def test_a_line_of_more_than_2_to_the_53_quarters_is_refused(T, B, width, H, G):
    """Sizes up to the last doubling that fits are taken, and no more."""
    def status(scale):
        s = paged(tokens=T, requests=B, width=width * scale // 16, heads=H, kv_heads=G, q_stride=H * 64, head_dim=64)
        return bool(_paged._entries["svdq_paged_attention_workspace_bytes"](ctypes.byref(s))), call_paged(_paged._entries, s)
    taken = []
    scale = 16
    while scale * width <= 1 << 30:
        most = longest(T, width * scale // 16 * 16, B, H, G)
        sized, code = status(scale)
        assert sized == (most <= 2.0 ** 51) and (code == SHAPE) == (most > 2.0 ** 51)
        taken.append(sized)
        scale *= 2
    assert not all(taken)


def test_packed_calls_count_in_whole_numbers():
    """(as many as 2^52 of them)"""
    for T, B in ((1 << 20, 4), (1 << 25, 1 << 10), (1 << 26, 16), (1 << 27, 1)):
        s = packed(tokens_q=T, tokens_k=T, sequences=B, heads=8, kv_heads=4, head_dim=64)
        want = longest(T, T, B, 8, 4) <= 2.0 ** 52
        assert (call_packed(_paged._entries, s) == SHAPE) == (not want)
    assert call_packed(_paged._entries, packed(sequences=0)) == OK


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("B,works", [(20, True), (200, False)])
def test_starts_that_descend_again_and_again(B, works, causal):
    """Every second sequence has all rows.  The line of 200 (100 times 50 tiles) is longer than that
    of any ascending starts, and no row is written; that of 20 is not, and the rows hold the result
    that all of them have."""
    T, H, D, R = 6400, 1, 64, 128
    g = torch.Generator(device="cuda").manual_seed(3)
    q, k, v = (torch.randn(T, H, D, generator=g, device="cuda").to(BF) for _ in range(3))
    n = T // R
    each = n * (256 + R) + R * n * (n - 1) // 2 if causal else n * (T + 256)
    assert (B // 2 * each <= longest(T, T, B, 1, 1)) == works
    at = torch.tensor([T * (i % 2) for i in range(B + 1)], dtype=torch.int32, device="cuda")
    buf = torch.full((T, H, D), -777.0, dtype=BF, device="cuda")
    out = bdt.packed_attention(q, k, v, at, causal=causal, out=buf)
    if works:
        from tests.test_gpu_paged import check, sequence_64
        check(out, *sequence_64(q, k, v, D ** -0.5, causal), "rows of %d sequences" % (B // 2))
    else:
        assert bool((out == -777).all())

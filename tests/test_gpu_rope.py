"""Rotary tables with several axes and the Q / K norm and turn, against 64-bit plain forms.

Tolerances (u = 2^-24, the half step of fp32):
- tables: the reduced angle in half turns, at most 1, is rounded to fp32 (moves the angle by
  at most pi u), the fp32 sine and cosine are within 2 ulp (4 u at magnitude 1); the 64-bit
  angle of a position up to 2^21 is off by less than 2^21 2^-51: together below 8 u = 2^-21.
- norm and turn: at most 16 fp32 roundings (12 in the sum of squares, halved by the root;
  root, quotient, gain, two products, one sum) of a pair's terms, 16 u (|a| + |b|), and the
  one rounding to bf16, 2^-8 relative.
"""
import numpy as np
import pytest
import torch

import bit_diffusion_transformer_amd as bdt
from bit_diffusion_transformer_amd import _attention
from tests.helpers import DEV, bf16_host

pytestmark = pytest.mark.gpu

AXES = [((16, 56, 56), 10000.0), ((44, 42, 42), 256.0), ((64,), 1e6), ((2, 2, 4), 10000.0),
        ((32, 32, 32, 32), (100.0, 1e3, 1e4, 1e5)), ((128, 128), 10000.0), ((8, 28, 28), 10000.0)]


def tables_64(pos, dims, theta):
    thetas = [theta] * len(dims) if np.isscalar(theta) else theta
    cols = [pos[:, a:a + 1].astype(np.float64) * np.float64(t) ** (-2.0 * np.arange(d // 2) / d)
            for a, (d, t) in enumerate(zip(dims, thetas))]
    angle = np.concatenate(cols, axis=1)
    return np.cos(angle), np.sin(angle)


@pytest.mark.parametrize("dims,theta", AXES, ids=lambda v: str(v).replace(" ", ""))
@pytest.mark.parametrize("S", [1, 2, 77, 1031, 70001])
def test_tables(dims, theta, S):
    rng = np.random.default_rng(S + len(dims))
    pos = rng.integers(0, 1 << 21, (S, len(dims))).astype(np.float32)
    pos[::3] = rng.uniform(-50, 50, pos[::3].shape)          # fractional and negative ones
    pos[0] = 0.0
    cos, sin = bdt.rope_tables(torch.from_numpy(pos).to(DEV), dims, theta)
    c, s = tables_64(pos, dims, theta)
    assert cos.shape == c.shape and cos.is_contiguous() and sin.is_contiguous()
    assert np.all(cos[0].cpu().numpy() == 1.0) and np.all(sin[0].cpu().numpy() == 0.0)
    assert np.abs(cos.cpu().numpy() - c).max() <= 2.0 ** -21
    assert np.abs(sin.cpu().numpy() - s).max() <= 2.0 ** -21


def turn_64(qkv, B, S, H, D, gq, gk, eps, cos, sin):
    """(Q, K, V) in 64 bits and, per element, |a| + |b| of its pair before the turn."""
    x = qkv.double().cpu().view(B, S, 3, H, D).permute(2, 0, 3, 1, 4)
    cos, sin = cos.double().cpu(), sin.double().cpu()
    out, mag = [], []
    for sec, g in ((0, gq), (1, gk)):
        y = x[sec]
        if g is not None:
            y = y / torch.sqrt(y.square().mean(-1, keepdim=True) + eps) * g.double().cpu()
        a, b = y[..., 0::2], y[..., 1::2]
        out.append(torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2))
        mag.append((a.abs() + b.abs()).repeat_interleave(2, dim=-1))
    return out, mag, x[2]


def _inputs(B, S, H, D, norm, seed):
    g = torch.Generator().manual_seed(seed)
    qkv = (torch.randn(B * S, 3 * H * D, generator=g) * 3).to(torch.bfloat16)
    gq, gk = [(1 + 0.3 * torch.randn(D, generator=g)).to(torch.bfloat16) for _ in range(2)]
    pos = torch.randint(0, 5000, (S, 2), generator=g).float()
    cos, sin = bdt.rope_tables(pos.to(DEV), (D // 2, D // 2))
    on = lambda t: None if t is None else t.to(DEV)   # noqa: E731
    return on(qkv), on(gq if norm in ("both", "q") else None), \
        on(gk if norm in ("both", "k") else None), cos, sin


def _check(Q, K, ref, mag, what):
    for name, got, want, m in (("Q", Q, ref[0], mag[0]), ("K", K, ref[1], mag[1])):
        err = (got.double().cpu() - want).abs()
        tol = 2.0 ** -8 * want.abs() + 16 * 2.0 ** -24 * m
        assert bool((err <= tol).all()), "%s %s: worst %.3g of the bound" % (
            what, name, float((err / tol.clamp_min(1e-300)).max()))


@pytest.mark.parametrize("B,S,H,D", [(1, 1, 1, 128), (1, 1, 2, 64), (1, 96, 24, 128), (3, 50, 18, 64),
                                     (5, 7, 3, 128), (130, 1, 2, 64), (2, 1031, 4, 128),
                                     (1, 333, 2, 64)])
@pytest.mark.parametrize("norm", ["both", "none", "q", "k"])
def test_norm_and_turn(B, S, H, D, norm):
    qkv, gq, gk, cos, sin = _inputs(B, S, H, D, norm, 7 * S + H)
    Q, K, V = bdt.qkv_norm_rope(qkv, H, D, S, gq, gk, 1e-6, cos, sin)
    ref, mag, v = turn_64(qkv, B, S, H, D, gq, gk, 1e-6, cos, sin)
    _check(Q, K, ref, mag, "B%d S%d H%d D%d %s" % (B, S, H, D, norm))
    assert torch.equal(V.double().cpu(), v)


def test_zero_rows_and_outputs_stay_inside():
    """All-zero heads give zeros (eps > 0), and nothing is written outside Q, K and V."""
    B, S, H, D = 2, 37, 2, 64
    qkv, gq, gk, cos, sin = _inputs(B, S, H, D, "both", 3)
    qkv[5] = 0
    n = B * S * H * D
    bufs = [torch.full((n + 256,), -777.0, dtype=torch.bfloat16, device=DEV) for _ in range(3)]
    q, k, v = (b[128:128 + n].view(B, H, S, D) for b in bufs)
    epi = bdt.qkv_epilogue(H, D, S, gq, gk, 1e-6, cos, sin, q, k, v)
    _attention.svdq_qkv_norm_rope(qkv, B * S, epi)
    Q, K, V = bdt.qkv_norm_rope(qkv, H, D, S, gq, gk, 1e-6, cos, sin)
    for b, t in zip(bufs, (Q, K, V)):
        assert bool((b[:128] == -777).all()) and bool((b[128 + n:] == -777).all())
        assert torch.equal(b[128:128 + n].view_as(t), t)
        assert bool((t[0, :, 5] == 0).all())


def test_turn_equals_the_fused_epilogue_of_the_4bit_gemm():
    """linear_qkv against the plain 4-bit layer's [M, N] output followed by qkv_norm_rope: the
    same function, apart from the projection's own rounding to bf16 (2^-8 of each element before
    norm and turn; the norm's denominator moves by as much again) and the output's."""
    from synth import LayerSpec, make_layer
    from tests.helpers import to_dev
    B, S, H, D, K, r = 2, 80, 2, 128, 320, 32
    L = make_layer(LayerSpec("t", B * S, K, 3 * H * D, r, 0.01, 20.0, 4, False, act=0, bias=True,
                             cfg_id=390))
    _, gq, gk, cos, sin = _inputs(B, S, H, D, "both", 11)
    qw, sw = bdt.pack_weights(to_dev(L.R))
    args = (to_dev(L.X), to_dev(L.lam), to_dev(L.L1), qw, sw, to_dev(L.L2), to_dev(L.bias))
    bdt.svdq_debug_set_tile_policy(bdt.TILES_FULL)
    try:
        fused = bdt.linear_qkv(*args, H, D, S, gq, gk, 1e-6, cos, sin)
        Y = bdt.linear(*args)
    finally:
        bdt.svdq_debug_set_tile_policy(bdt.TILES_AUTO)
    apart = bdt.qkv_norm_rope(Y, H, D, S, gq, gk, 1e-6, cos, sin)
    assert torch.equal(fused[2], apart[2])
    _, mag, _ = turn_64(Y, B, S, H, D, gq, gk, 1e-6, cos, sin)
    for f, a, m in zip(fused[:2], apart[:2], mag):
        err = (f.double() - a.double()).abs().cpu()
        # one 2^-8 of the pair for the projection's rounding, one for the norm, one for each
        # output; their products, 2^-8 of that again, and the fp32 steps: below 0.1 more
        assert bool((err <= 4.1 * 2.0 ** -8 * m).all())


def test_tables_feed_the_fused_epilogue_and_replay_in_a_graph():
    """Captured and replayed, on a stream of its own, with new inputs between the replays."""
    B, S, H, D = 1, 61, 2, 128
    qkv, gq, gk, cos, sin = _inputs(B, S, H, D, "both", 5)
    pos = torch.arange(S * 2, dtype=torch.float32, device=DEV).view(S, 2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(2):
            c, n = bdt.rope_tables(pos, (64, 64))
            bdt.qkv_norm_rope(qkv, H, D, S, gq, gk, 1e-6, c, n)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c, n = bdt.rope_tables(pos, (64, 64))
        Q, K, V = bdt.qkv_norm_rope(qkv, H, D, S, gq, gk, 1e-6, c, n)
    for it in range(4):
        pos += 3.0
        qkv.mul_(-0.5)
        g.replay()
        torch.cuda.synchronize()
        c2, n2 = bdt.rope_tables(pos, (64, 64))
        want = bdt.qkv_norm_rope(qkv, H, D, S, gq, gk, 1e-6, c2, n2)
        for a, b in zip((Q, K, V), want):
            assert np.array_equal(bf16_host(a), bf16_host(b)), "replay %d" % it


def test_empty():
    cos, sin = bdt.rope_tables(torch.empty(0, 2, device=DEV), (64, 64))
    assert cos.shape == (0, 64)
    t = torch.zeros(4, 64, device=DEV)
    Q, _, _ = bdt.qkv_norm_rope(torch.empty(0, 768, dtype=torch.bfloat16, device=DEV), 2, 128, 4,
                                None, None, 1e-6, t, t)
    assert Q.shape == (0, 2, 4, 128)

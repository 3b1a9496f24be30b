"""The attention half of a block, its operators run together: rotary tables of a text + image
sequence, the QKV projection (W4A4 with the fused epilogue, or 8-bit followed by the norm and
turn), sparse attention over a padded batch, the output projection."""
import pytest
import torch

import bit_diffusion_transformer_amd as bdt
from synth import LayerSpec, make_layer
from tests.helpers import DEV, to_dev
from tests.test_gpu_i8 import check_y, y_64
from tests.test_gpu_rope import _check as check_turn, turn_64
from tests.test_gpu_sparse_attention import attention_64, check, lists_64

pytestmark = pytest.mark.gpu

B, TEXT, GRID, H, D, K = 2, 70, (1, 18, 20), 4, 64, 192
S = TEXT + GRID[0] * GRID[1] * GRID[2]
M, HD = B * S, H * D
KEEP, FIRST, LENS = 4, 2, [S, S - 77]


def _tables():
    t, h, w = torch.meshgrid(*[torch.arange(n) for n in GRID], indexing="ij")
    pos = torch.zeros(S, 3)
    pos[:TEXT, 0] = torch.arange(TEXT)
    pos[TEXT:] = torch.stack([t, h, w], -1).view(-1, 3)
    return bdt.rope_tables(pos.to(DEV), (16, 24, 24))


def _gammas():
    g = torch.Generator().manual_seed(2)
    return [(1 + 0.2 * torch.randn(D, generator=g)).to(torch.bfloat16).to(DEV) for _ in range(2)]


def _w4a4(n_in, n_out, cid):
    L = make_layer(LayerSpec("c%d" % cid, M, n_in, n_out, 16, 0.01, 20.0, 4, False, act=0, bias=True,
                             cfg_id=400 + cid))
    qw, sw = bdt.pack_weights(to_dev(L.R))
    return L, dict(lam=to_dev(L.lam), L1=to_dev(L.L1), qw=qw, sw=sw, L2=to_dev(L.L2),
                   bias=to_dev(L.bias))


def _graph(fn, replays, X, inputs, want):
    """fn() captured, replayed on changed inputs, compared with the eager results."""
    fn()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        Y = fn()
    for it in range(replays):
        X.copy_(inputs[it % 2])
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(Y, want[it % 2]), "replay %d" % it


def test_w4a4_attention():
    Lq, qkv = _w4a4(K, 3 * HD, 1)
    _, out = _w4a4(HD, 128, 2)
    cos, sin = _tables()
    gq, gk = _gammas()
    kv_len = torch.tensor(LENS, dtype=torch.int32, device=DEV)
    X = to_dev(Lq.X)

    def run():
        return bdt.attention(X, qkv, out, H, D, S, gq, gk, 1e-6, cos, sin, KEEP, FIRST, kv_len)
    Y = run()
    assert Y.shape == (M, 128)
    # the same steps one by one, the attention against 64 bits
    Q, Kt, V = bdt.linear_qkv(X, qkv["lam"], qkv["L1"], qkv["qw"], qkv["sw"], qkv["L2"], qkv["bias"],
                              H, D, S, gq, gk, 1e-6, cos, sin)
    A, blocks = bdt.sparse_attention(Q, Kt, V, KEEP, FIRST, kv_len=kv_len, return_blocks=True)
    assert torch.equal(blocks.cpu(), lists_64(Q, Kt, LENS, KEEP, FIRST))
    ref, tol = attention_64(Q, Kt, V, blocks.cpu(), D ** -0.5, LENS)
    check(A, ref, tol, "attention of the chain")
    assert torch.equal(Y, bdt.linear(A.view(M, HD), out["lam"], out["L1"], out["qw"], out["sw"],
                                     out["L2"], out["bias"]))
    X0, X1 = X.clone(), X.flip(0).contiguous()
    X.copy_(X1)
    want = [Y, run()]
    _graph(run, 4, X, [X0, X1], want)


def test_8bit_attention():
    g = torch.Generator(device=DEV).manual_seed(8)

    def rn(*s):
        return torch.randn(s, generator=g, device=DEV)
    X, lam = rn(M, K).to(torch.bfloat16), 0.5 + torch.rand(K, generator=g, device=DEV)
    qw, sw = bdt.i8_pack_weights(rn(3 * HD, K) * K ** -0.5 * lam)
    ow, os = bdt.i8_pack_weights(rn(128, HD) * HD ** -0.5)
    bias = rn(3 * HD).to(torch.bfloat16)
    cos, sin = _tables()
    gq, gk = _gammas()
    kv_len = torch.tensor(LENS, dtype=torch.int32, device=DEV)

    def run(steps=None):
        P = bdt.i8_linear(X, lam, qw, sw, bias)
        Q, Kt, V = bdt.qkv_norm_rope(P, H, D, S, gq, gk, 1e-6, cos, sin)
        A, blocks = bdt.sparse_attention(Q, Kt, V, KEEP, FIRST, kv_len=kv_len, return_blocks=True)
        Y = bdt.i8_linear(A.view(M, HD), None, ow, os)
        if steps is not None:
            steps.extend((P, Q, Kt, V, A, blocks))
        return Y
    steps = []
    Y = run(steps)
    P, Q, Kt, V, A, blocks = steps
    qa, sa = bdt.i8_quantize_act(X, lam)
    ref, mag = y_64(qa, sa, qw, sw, bias, 0)
    check_y(P, ref, mag, 0, "projection")
    ref, mag, v = turn_64(P, B, S, H, D, gq, gk, 1e-6, cos, sin)
    check_turn(Q, Kt, ref, mag, "turn")
    assert torch.equal(V.double().cpu(), v)
    assert torch.equal(blocks.cpu(), lists_64(Q, Kt, LENS, KEEP, FIRST))
    ref, tol = attention_64(Q, Kt, V, blocks.cpu(), D ** -0.5, LENS)
    check(A, ref, tol, "attention")
    qa, sa = bdt.i8_quantize_act(A.view(M, HD))
    ref, mag = y_64(qa, sa, ow, os, None, 0)
    check_y(Y, ref, mag, 0, "output projection")
    X0, X1 = X.clone(), X.flip(0).contiguous()
    X.copy_(X1)
    want = [Y, run()]
    _graph(run, 4, X, [X0, X1], want)

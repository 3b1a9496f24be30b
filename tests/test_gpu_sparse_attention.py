"""Block selection and block-sparse attention against 64-bit plain forms.

Lists have to be equal: means and scores are 64-bit on both sides, and the inputs' scores
differ by far more than 2^-50 (or are exactly equal: small whole numbers, whose 64-bit sums
are exact).

Outputs.  With p the exact weights and w = sum p |v|:
- a score's fp32 sum of D exact products is off by at most (D + 8) 2^-23 scale sum |q k| =: d
  (the + 8: the product with the scale and the maximum, and the exponent's own rounding), so a
  weight by a factor within 1 +- d (1 + small), and the normalized one within 1 +- 2 d;
- each weight is rounded to bf16 for the second product: 2^-8 of it;
- fp32 sums over n keys of weights and of weighted values: 2 n 2^-23 of w;
- 2^-12 for the exponential, the reciprocal, a change of the running maximum, and products of
  the terms above; one rounding of the result to bf16: 2^-8 of it.
"""
import numpy as np
import pytest
import torch

import bit_diffusion_transformer_amd as bdt
from bit_diffusion_transformer_amd import _attention
from tests.helpers import DEV

pytestmark = pytest.mark.gpu
QB, KB = 128, 64


def lens_of(kv_len, B, Sk):
    return [Sk] * B if kv_len is None else [min(max(int(n), 0), Sk) for n in kv_len]


def lists_64(q, k, kv_len, keep, first):
    B, H, Sq, D = q.shape
    G, Sk = k.shape[1:3]
    nq = -(-Sq // QB)
    out = torch.full((B, H, nq, keep), -1, dtype=torch.int32)
    for b, n in enumerate(lens_of(kv_len, B, Sk)):
        nk = -(-n // KB)
        if nk == 0:
            continue
        for h in range(H):
            kd = torch.zeros(nk * KB, D, dtype=torch.float64, device=q.device)
            kd[:n] = k[b, h // (H // G), :n].double()
            kc = torch.full((nk, 1), KB, dtype=torch.float64, device=q.device)
            kc[-1] = n - (nk - 1) * KB
            km = kd.view(nk, KB, D).sum(1) / kc
            qd = torch.zeros(nq * QB, D, dtype=torch.float64, device=q.device)
            qd[:Sq] = q[b, h].double()
            qc = torch.full((nq, 1), QB, dtype=torch.float64, device=q.device)
            qc[-1] = Sq - (nq - 1) * QB
            score = (qd.view(nq, QB, D).sum(1) / qc) @ km.t()
            score[:, :first] = np.inf
            order = torch.sort(score, dim=1, descending=True, stable=True).indices[:, :keep]
            out[b, h, :, :order.shape[1]] = order.sort(1).values.to(torch.int32).cpu()
    return out


def usable(lst, n):
    """The entries of a list that count, by the documented rule."""
    got, top = [], -1
    for e in lst:
        if 0 <= e < -(-n // KB) and e > top:
            got.append(e)
        top = max(top, e)
    return got


def attention_64(q, k, v, lists, scale, kv_len, planes=None):
    """(out, tolerance) fp64 [B, Sq, H, D] on the GPU, over the given (b, h) (default all)."""
    B, H, Sq, D = q.shape
    G, Sk = k.shape[1:3]
    out = torch.zeros(B, Sq, H, D, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    lens = lens_of(kv_len, B, Sk)
    for b in range(B):
        for h in range(H):
            if planes is not None and (b, h) not in planes:
                continue
            for i in range(-(-Sq // QB)):
                keys = [n for e in usable(lists[b, h, i].tolist(), lens[b])
                        for n in range(e * KB, min((e + 1) * KB, lens[b]))]
                if not keys:
                    continue
                idx = torch.tensor(keys, device=q.device)
                rows = slice(i * QB, min((i + 1) * QB, Sq))
                qd = q[b, h, rows].double()
                kd, vd = k[b, h // (H // G), idx].double(), v[b, h // (H // G), idx].double()
                p = torch.softmax(scale * (qd @ kd.t()), dim=1)
                o, w = p @ vd, p @ vd.abs()
                d = (D + 8) * 2.0 ** -23 * scale * (qd.abs() @ kd.abs().t()).amax(1, keepdim=True)
                out[b, rows, h] = o
                tol[b, rows, h] = 2.0 ** -8 * o.abs() + w * (
                    2 * d + 2.0 ** -8 + 2 * len(keys) * 2.0 ** -23 + 2.0 ** -12)
    return out, tol


def inputs(B, H, G, D, Sq, Sk, seed, gain=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def r(*s):
        return torch.randn(s, generator=g, device=DEV)
    theme = r(B, G, -(-max(Sq, Sk) // 40), D)
    q = theme.repeat_interleave(H // G, 1).repeat_interleave(40, 2)[:, :, :Sq] + r(B, H, Sq, D)
    k = theme.repeat_interleave(40, 2)[:, :, :Sk] + r(B, G, Sk, D)
    return (gain * q).to(torch.bfloat16), k.to(torch.bfloat16), r(B, G, Sk, D).to(torch.bfloat16)


def check(out, ref, tol, what):
    err = (out.double() - ref).abs()
    assert bool(torch.isfinite(out.float()).all()), "%s: not finite" % what
    assert bool((err <= tol + 1e-30).all()), "%s: worst %.3g of the bound" % (
        what, float((err / (tol + 1e-30)).max()))


# B, H, G, D, Sq, Sk, keep, first, kv_len
CASES = [
    (1, 1, 1, 128, 1, 1, 1, 0, None),
    (1, 2, 1, 64, 1, 63, 2, 1, None),
    (2, 2, 2, 128, 127, 64, 1, 0, [64, 1]),
    (1, 4, 2, 64, 128, 65, 3, 0, [65]),
    (2, 3, 3, 128, 129, 1000, 4, 2, [999, 0]),
    (3, 2, 1, 64, 300, 640, 5, 0, [640, 385, -7]),
    (2, 4, 1, 128, 257, 777, 100, 3, [5000, 321]),
    (1, 6, 6, 128, 1000, 1000, 6, 6, None),
    (1, 2, 2, 64, 2048, 2048, 9, 0, None),
    (4, 8, 2, 128, 1, 5000, 20, 1, [5000, 4999, 1281, 64]),        # few query blocks: split
    (1, 2, 2, 64, 5, 9000, 130, 0, [8970]),
    (1, 1, 1, 128, 130, 4096, 64, 0, None),                        # every block
    (1, 2, 1, 128, 200, 40000, 10, 2, [39950]),                    # 625 key blocks
    (1, 1, 1, 64, 150, 70000, 33, 0, None),                        # 1094
    (1, 1, 1, 64, 140, 140001, 7, 1, None),                        # 2188
    (1, 1, 1, 64, 3, 1 << 18, 70, 0, None),                        # the longest
    (2, 16, 16, 64, 1200, 1200, 4, 1, [1200, 700]),
    (1, 24, 24, 128, 1500, 1500, 7, 2, None),
]


@pytest.mark.parametrize("B,H,G,D,Sq,Sk,keep,first,kv", CASES)
def test_sparse_attention(B, H, G, D, Sq, Sk, keep, first, kv):
    q, k, v = inputs(B, H, G, D, Sq, Sk, Sq + Sk)
    kv_len = None if kv is None else torch.tensor(kv, dtype=torch.int32, device=DEV)
    for b, n in enumerate(lens_of(kv, B, Sk)):                     # masked places hold anything
        k[b, :, n:] = float("nan")
        v[b, :, n:] = float("inf")
        v[b, :, n:, ::2] = float("nan")
    out, blocks = bdt.sparse_attention(q, k, v, keep, first=first, kv_len=kv_len, return_blocks=True)
    assert out.shape == (B, Sq, H, D)
    want = lists_64(q, k, kv, keep, first)
    assert torch.equal(blocks.cpu(), want)
    assert torch.equal(bdt.select_blocks(q, k, keep, first, kv_len), blocks)
    ref, tol = attention_64(q, k, v, want, D ** -0.5, kv)
    check(out, ref, tol, "sparse_attention")
    for b, n in enumerate(lens_of(kv, B, Sk)):
        if n == 0:
            assert bool((out[b] == 0).all())
    assert torch.equal(bdt.block_attention(q, k, v, blocks, kv_len=kv_len), out)
    assert torch.equal(bdt.sparse_attention(q, k, v, keep, first=first, kv_len=kv_len), out)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Sk,keep,first", [(640, 3, 0), (640, 3, 1), (9000, 40, 2), (70000, 5, 0)])
def test_equal_scores_go_to_the_lowest_number(D, Sk, keep, first):
    """Whole numbers: sums and products are exact in 64 bits.  Three kinds of blocks only, so
    nearly every score is shared; the last block (of fewer keys) has the same mean."""
    q = torch.ones(1, 2, 200, D, dtype=torch.bfloat16, device=DEV)
    q[:, 1] = -1
    nk = -(-Sk // KB)
    kind = torch.randint(0, 3, (nk,), generator=torch.Generator().manual_seed(Sk + keep)).float() - 1
    k = kind.repeat_interleave(KB)[:Sk].to(DEV).to(torch.bfloat16)[None, None, :, None]
    k = k.expand(1, 1, Sk, D).contiguous()
    blocks = bdt.select_blocks(q, k, keep, first)
    assert torch.equal(blocks.cpu(), lists_64(q, k, None, keep, first))
    k.zero_()                                                      # all equal, and -0 == +0
    k[:, :, KB:2 * KB] = -0.0
    blocks = bdt.select_blocks(q, k, keep, first)
    assert blocks.cpu().tolist() == [[[list(range(keep))] * 2] * 2]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Sq", [1, 300])
def test_given_lists_are_read_by_the_documented_rule(D, Sq):
    """Repeated, descending, negative and far too large entries, empty lists, in the middle of
    others; with and without the split over keys."""
    B, H, G, Sk, kv = 2, 2, 1, 1500, [1500, 700]
    q, k, v = inputs(B, H, G, D, Sq, Sk, 5)
    kv_len = torch.tensor(kv, dtype=torch.int32, device=DEV)
    nq, keep = -(-Sq // QB), 70
    rng = np.random.default_rng(3)
    lists = torch.from_numpy(np.sort(rng.integers(-3, 30, (B, H, nq, keep)), axis=-1).astype(np.int32))
    lists[0, 0, 0] = torch.from_numpy(rng.integers(-5, 2 ** 31 - 1, keep).astype(np.int32))
    lists[0, 0, 0, :4] = torch.tensor([4, 4, 3, 9])
    lists[0, 1, 0] = -1
    lists[0, 1, 0, 66] = 7                                         # behind 66 empty entries
    lists[1, 1, 0] = -2 ** 31
    lists[1, 0, 0] = 2 ** 31 - 1
    out = bdt.block_attention(q, k, v, lists.to(DEV), scale=0.3, kv_len=kv_len)
    ref, tol = attention_64(q, k, v, lists, 0.3, kv)
    check(out, ref, tol, "given lists")
    assert bool((out[1, :QB] == 0).all())


@pytest.mark.parametrize("H,G,D,Sq,Sk,keep", [
    (40, 1, 128, 3, 700, 5),           # more heads per K head than a workgroup has groups of threads
    (35, 1, 64, 1, 1300, 9),
    (6, 2, 128, 16, 2000, 7), (6, 2, 128, 17, 2000, 7),
    (17, 1, 64, 8, 900, 4), (17, 1, 64, 9, 900, 4),
    (2, 2, 64, 127, 320, 2), (2, 2, 64, 1, 64, 1),
])
def test_few_queries(H, G, D, Sq, Sk, keep):
    """One query block, from one row to nearly all of it; a sequence that ends inside a key
    block and one without keys."""
    kv = [Sk - 1, 0, Sk]
    q, k, v = inputs(3, H, G, D, Sq, Sk, Sq + H)
    kv_len = torch.tensor(kv, dtype=torch.int32, device=DEV)
    k[0, :, Sk - 1] = float("nan")
    out, blocks = bdt.sparse_attention(q, k, v, keep, first=1, kv_len=kv_len, return_blocks=True)
    want = lists_64(q, k, kv, keep, 1)
    assert torch.equal(blocks.cpu(), want)
    ref, tol = attention_64(q, k, v, want, D ** -0.5, kv)
    check(out, ref, tol, "few queries")
    ones, kind = torch.ones_like(q), torch.arange(Sk, device=DEV) // KB % 2      # many ties
    alike = kind.to(torch.bfloat16)[None, None, :, None].expand_as(k).contiguous()
    same = bdt.select_blocks(ones, alike, keep)
    assert torch.equal(same.cpu(), lists_64(ones, alike, None, keep, 0))


@pytest.mark.parametrize("gain", [0.0, 40.0, 4000.0])
@pytest.mark.parametrize("Sq", [2, 400])
def test_extreme_scores(gain, Sq):
    """All scores zero; scores in the thousands (one key takes nearly all; the running maximum
    moves often)."""
    B, H, G, D, Sk, keep = 1, 3, 3, 128, 2000, 16
    q, k, v = inputs(B, H, G, D, Sq, Sk, 9, gain)
    k = k * torch.linspace(0.1, 2.0, Sk, device=DEV).to(torch.bfloat16)[None, None, :, None]
    out, blocks = bdt.sparse_attention(q, k, v, keep, return_blocks=True)
    assert torch.equal(blocks.cpu(), lists_64(q, k, None, keep, 0))
    ref, tol = attention_64(q, k, v, blocks.cpu(), D ** -0.5, None)
    check(out, ref, tol, "gain %g" % gain)


def test_dense_when_every_block_is_kept():
    q, k, v = inputs(1, 2, 2, 64, 700, 700, 21)
    a = bdt.sparse_attention(q, k, v, 11)
    b = bdt.sparse_attention(q, k, v, 200, first=50)
    assert torch.equal(a, b)
    s = torch.softmax(q.double() @ k.double().transpose(2, 3) / 8.0, -1) @ v.double()
    ref, tol = attention_64(q, k, v, torch.arange(11).expand(1, 2, 6, 11), 0.125, None)
    assert float((s.permute(0, 2, 1, 3) - ref).abs().max()) < 1e-9
    check(a, ref, tol, "dense")


@pytest.mark.parametrize("B,H,G,D,Sq,Sk,keep", [(1, 2, 1, 128, 200, 300, 3), (2, 4, 2, 64, 1, 3000, 30)])
def test_outputs_stay_inside(B, H, G, D, Sq, Sk, keep):
    q, k, v = inputs(B, H, G, D, Sq, Sk, 1)
    s = _attention._shape(q, k, None, keep, 0)
    n, nl = B * Sq * H * D, B * H * -(-Sq // QB) * keep
    buf = torch.full((n + 512,), -777.0, dtype=torch.bfloat16, device=DEV)
    lbuf = torch.full((nl + 512,), -99, dtype=torch.int32, device=DEV)
    need = bdt.svdq_sparse_attention_workspace_bytes(s)
    ws = torch.full((need + 512,), 0x5A, dtype=torch.uint8, device=DEV)
    lists = lbuf[256:256 + nl]
    bdt.svdq_sparse_attention(q, k, v, None, s, D ** -0.5, lists, buf[256:256 + n], ws[256:], need)
    assert bool((buf[:256] == -777).all()) and bool((buf[256 + n:] == -777).all())
    assert bool((lbuf[:256] == -99).all()) and bool((lbuf[256 + nl:] == -99).all())
    assert bool((ws[:256] == 0x5A).all()) and bool((ws[256 + need:] == 0x5A).all())
    out, blocks = bdt.sparse_attention(q, k, v, keep, return_blocks=True)
    assert torch.equal(buf[256:256 + n].view_as(out), out)
    assert torch.equal(lists.view_as(blocks), blocks)


@pytest.mark.parametrize("H,D,Sq,Sk,keep", [(3, 128, 500, 500, 4), (2, 64, 1, 4000, 40)])
def test_in_a_graph_and_on_two_streams(H, D, Sq, Sk, keep):
    q, k, v = inputs(1, H, H, D, Sq, Sk, 1)
    q2, k2, v2 = inputs(1, H, H, D, Sq, Sk, 2)
    want = [bdt.sparse_attention(a, b, c, keep, return_blocks=True) for a, b, c in ((q, k, v), (q2, k2, v2))]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        got = []
        for s, (a, b, c) in zip(streams, ((q, k, v), (q2, k2, v2))):
            with torch.cuda.stream(s):
                got.append(bdt.sparse_attention(a, b, c, keep, return_blocks=True))
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])
    qg, kg, vg = q.clone(), k.clone(), v.clone()
    kv_len = torch.full((1,), Sk, dtype=torch.int32, device=DEV)
    with torch.cuda.stream(streams[0]):
        bdt.sparse_attention(qg, kg, vg, keep, kv_len=kv_len)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, blocks = bdt.sparse_attention(qg, kg, vg, keep, kv_len=kv_len, return_blocks=True)
    for it in range(5):
        for dst, src in ((qg, (q, q2)), (kg, (k, k2)), (vg, (v, v2))):
            dst.copy_(src[it % 2])
        n = Sk if it < 3 else Sk // 3                              # a length read at replay
        kv_len.fill_(n)
        g.replay()
        torch.cuda.synchronize()
        w = want[it % 2] if n == Sk else bdt.sparse_attention(qg, kg, vg, keep, kv_len=kv_len,
                                                              return_blocks=True)
        assert torch.equal(out, w[0]) and torch.equal(blocks, w[1]), "replay %d" % it


def test_offsets_past_32_bits():
    """K and V of more than 2^31 elements; the last head is the one compared."""
    G, Sk, D, keep = 130, 1 << 18, 64, 3
    k = torch.zeros(1, G, Sk, D, dtype=torch.bfloat16, device=DEV)
    assert k.numel() > 1 << 31
    g = torch.Generator(device=DEV).manual_seed(4)
    k[0, G - 1] = torch.randn(Sk, D, generator=g, device=DEV).to(torch.bfloat16)
    q = torch.randn(1, G, 1, D, generator=g, device=DEV).to(torch.bfloat16)
    out, blocks = bdt.sparse_attention(q, k, k, keep, return_blocks=True)
    last = q[:, G - 1:].contiguous(), k[:, G - 1:].contiguous()
    want = lists_64(*last, None, keep, 0)
    assert torch.equal(blocks[:, G - 1:].cpu(), want)
    assert blocks[0, 0, 0].tolist() == [0, 1, 2]                    # all scores zero: the lowest
    ref, tol = attention_64(*last, last[1], want, D ** -0.5, None)
    check(out[:, :, G - 1:], ref, tol, "last head")


def test_empty():
    e = torch.empty(0, 2, 5, 64, dtype=torch.bfloat16, device=DEV)
    out, blocks = bdt.sparse_attention(e, e, e, 3, return_blocks=True)
    assert out.shape == (0, 5, 2, 64) and blocks.shape == (0, 2, 1, 3)
    q, k, v = inputs(1, 2, 2, 64, 1, 70, 1)
    assert bdt.sparse_attention(q[:, :, :0].contiguous(), k, v, 3).shape == (1, 0, 2, 64)

"""The operators of a paged cache run together, as a server runs them: page tables from request
lengths, the projection with its norm and turn into the cache, attention over the cache; prompts
in chunks, single tokens, requests that end and hand back their pages; and the whole half block
on W4A4 layers."""
import numpy as np
import pytest
import torch

import bit_diffusion_transformer_amd as bdt
from synth import LayerSpec, make_layer
from tests.helpers import DEV, to_dev
from tests.test_gpu_paged import check, ints, normal, sequence_64, starts_of

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
EPS = 1e-6


def rope(P, R):
    return bdt.rope_tables(torch.arange(P, dtype=torch.float32, device=DEV)[:, None].contiguous(), [R])


def turned(qkv, H, G, D, gq, gk, cos, sin, half):
    """Q [n, H, D], K and V [n, G, D] of one request's rows 0 .. n - 1, through a cache of its own."""
    n, page = qkv.shape[0], 256
    kc = torch.zeros(-(-n // page), G, page, D, dtype=BF, device=DEV)
    vc = torch.zeros_like(kc)
    at = torch.arange(n, dtype=torch.int32, device=DEV)
    q = bdt.qkv_norm_rope_cache(qkv, H, G, gq, gk, EPS, cos, sin, at, at, kc, vc, half=half)
    return q, kc.transpose(1, 2).reshape(-1, G, D)[:n], vc.transpose(1, 2).reshape(-1, G, D)[:n]


@pytest.mark.parametrize("H,G,D,R,page,half", [(8, 2, 128, 128, 16, True), (6, 6, 64, 32, 64, False),
                                               (28, 4, 64, 64, 32, True), (4, 1, 128, 64, 256, False)])
def test_requests_served_step_by_step(H, G, D, R, page, half):
    """Every step's rows equal the attention of the whole request so far, in 64 bits, and a prompt
    in one piece through packed_attention agrees with its chunks."""
    lens = [300, 1, 97, 40]                            # tokens of each request in the end
    steps = [[150, 1, 0, 33], [149, 0, 64, 1], [1, 0, 1, 1], [0, 0, 32, 1], [0, 0, 0, 4]]
    assert [sum(s[b] for s in steps) for b in range(4)] == lens
    pages, width = sum(-(-n // page) for n in lens) + 1, -(-max(lens) // page)
    cos, sin = rope(400, R)
    gq, gk = 1 + normal(1, D, gain=0.2), 1 + normal(2, D, gain=0.2)
    qkv = [normal(10 + b, n, (H + 2 * G) * D) for b, n in enumerate(lens)]
    whole = [turned(x, H, G, D, gq, gk, cos, sin, half) for x in qkv]
    free = np.random.default_rng(0).permutation(pages).tolist()
    tables = torch.full((4, width), -1, dtype=torch.int32, device=DEV)
    kc = torch.full((pages, G, page, D), float("nan"), dtype=BF, device=DEV)
    vc = torch.full_like(kc, float("inf"))
    cached = [0] * 4
    for new in steps:
        T = sum(new) + 3                               # rows behind the last request
        X = torch.cat([qkv[b][cached[b]:cached[b] + n] for b, n in enumerate(new)] + [normal(5, 3, (H + 2 * G) * D)])
        at, kv, slots, positions, counts = bdt.page_tables(ints(cached), ints(new), ints(free), tables, page, pages, T)
        q = torch.full((T, H, D), -333.0, dtype=BF, device=DEV)
        bdt.qkv_norm_rope_cache(X, H, G, gq, gk, EPS, cos, sin, positions, slots, kc, vc, half=half, out=q)
        buf = torch.full((T, H, D), -777.0, dtype=BF, device=DEV)
        bdt.paged_attention(q, kc, vc, tables, at, kv, max_new=max(new), out=buf)
        taken, lost = counts.tolist()
        assert lost == 0 and at.tolist() == starts_of(new)
        free = free[taken:]
        assert bool((q[-3:] == -333).all()) and bool((buf[-3:] == -777).all())
        for b, n in enumerate(new):
            rows, a, end = slice(at[b], at[b + 1]), cached[b], cached[b] + n
            Q, K, V = (x[:end] for x in whole[b])
            assert torch.equal(q[rows], Q[a:])
            ref, tol = sequence_64(Q, K, V, D ** -0.5, True)
            check(buf[rows], ref[a:], tol[a:], "request %d" % b)
        cached = [c + n for c, n in zip(cached, new)]
    assert cached == lens
    Q, K, V = (torch.cat([w[i] for w in whole]) for i in range(3))
    out = bdt.packed_attention(Q, K, V, ints(starts_of(lens)))
    for b, n in enumerate(lens):
        rows = slice(*starts_of(lens)[b:b + 2])
        ref, tol = sequence_64(*whole[b], D ** -0.5, True)
        check(out[rows], ref, tol, "prompt %d" % b)
    # the first request ends; its pages serve a new one, whose rows see none of the old keys
    old = tables[0, :-(-lens[0] // page)].tolist()
    n = min(200, len(old) * page)
    tables[0] = -1
    x = normal(77, n, (H + 2 * G) * D)
    at, kv, slots, positions, counts = bdt.page_tables(ints([0] + lens[1:]), ints([n, 0, 0, 0]), ints(old), tables,
                                                       page, pages, n)
    q = bdt.qkv_norm_rope_cache(x, H, G, gq, gk, EPS, cos, sin, positions, slots, kc, vc, half=half)
    got = bdt.paged_attention(q, kc, vc, tables, at, kv, max_new=n)
    Q, K, V = turned(x, H, G, D, gq, gk, cos, sin, half)
    assert torch.equal(q, Q)
    ref, tol = sequence_64(Q, K, V, D ** -0.5, True)
    check(got, ref, tol, "the new request")


def w4a4(n_in, n_out, cid):
    L = make_layer(LayerSpec("p%d" % cid, 64, n_in, n_out, 16, 0.01, 20.0, 4, False, act=0, bias=True, cfg_id=500 + cid))
    qw, sw = bdt.pack_weights(to_dev(L.R))
    return dict(lam=to_dev(L.lam), L1=to_dev(L.L1), qw=qw, sw=sw, L2=to_dev(L.L2), bias=to_dev(L.bias))


def test_half_block_over_a_cache():
    """cached_attention is its four calls, bit for bit, eager and replayed with other lengths."""
    H, G, D, K, page, pages = 6, 2, 64, 192, 32, 40
    qkv, out = w4a4(K, (H + 2 * G) * D, 1), w4a4(H * D, 128, 2)
    cos, sin = rope(500, D)
    gq, gk = 1 + normal(1, D, gain=0.2), None
    T, B = 70, 3
    X = normal(3, T, K)
    cached, new = ints([100, 0, 31]), ints([1, 64, 5])
    tables = torch.full((B, 8), -1, dtype=torch.int32, device=DEV)
    tables[0, :4] = ints([3, 9, 27, 1])
    tables[2, 0] = 0
    free = ints(list(range(30, 40)))
    caches = [normal(4, pages, G, page, D), normal(5, pages, G, page, D)]

    def one(kc, vc):
        at, kv, slots, positions, counts = bdt.page_tables(cached, new, free, tables, page, pages, T)
        return bdt.cached_attention(X, qkv, out, H, G, D, gq, gk, EPS, cos, sin, kc, vc, tables, at, kv, slots,
                                    positions, max_new=64, half=True)

    def four(kc, vc):
        at, kv, slots, positions, counts = bdt.page_tables(cached, new, free, tables, page, pages, T)
        P = bdt.linear(X, qkv["lam"], qkv["L1"], qkv["qw"], qkv["sw"], qkv["L2"], qkv["bias"])
        Q = bdt.qkv_norm_rope_cache(P, H, G, gq, gk, EPS, cos, sin, positions, slots, kc, vc, half=True)
        A = bdt.paged_attention(Q, kc, vc, tables, at, kv, max_new=64)
        return bdt.linear(A.view(T, H * D), out["lam"], out["L1"], out["qw"], out["sw"], out["L2"], out["bias"])
    a, b = [c.clone() for c in caches], [c.clone() for c in caches]
    assert torch.equal(one(*a), four(*b))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and not torch.equal(a[0], caches[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Y = one(*a)
    for it in range(4):
        X.copy_(normal(20 + it, T, K))
        new.copy_(ints([1 + it, 64 - it, 5]))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(Y, four(*b)), "replay %d" % it
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])

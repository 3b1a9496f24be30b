"""Attention of packed sequences and over a paged cache against 64-bit plain forms.

Outputs.  With p the exact weights and w = sum p |v|:
- a score's fp32 sum of D exact products is off by at most (D + 8) 2^-23 scale sum |q k| =: d
  (the + 8: the product with the scale and the maximum, and the exponent's own rounding), so a
  weight by a factor within 1 +- d (1 + small), and the normalized one within 1 +- 2 d;
- each weight is rounded to bf16 for the second product: 2^-8 of it;
- fp32 sums over n keys of weights and of weighted values: 2 n 2^-23 of w;
- 2^-12 for the exponential, the reciprocal, a change of the running maximum, the join of
  parts, and products of the terms above; one rounding of the result to bf16: 2^-8 of it.
"""
import numpy as np
import pytest
import torch

import bit_diffusion_transformer_amd as bdt
from tests.helpers import DEV

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def starts_of(lens):
    return [0] + np.cumsum(lens).tolist()


def sequence_64(q, k, v, scale, causal, dead=None):
    """(out, tolerance) fp64 [n, H, D] of one sequence: q [n, H, D], k, v [m, G, D]; dead [m]:
    keys that no row sees."""
    n, H, D = q.shape
    m, G = k.shape[:2]
    out = torch.zeros(n, H, D, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    if n == 0 or m == 0:
        return out, tol
    key = torch.arange(m, device=q.device)
    row = torch.arange(n, device=q.device)
    sees = key[None, :] <= row[:, None] + (m - n) if causal else torch.ones(n, m, dtype=torch.bool,
                                                                            device=q.device)
    if dead is not None:
        sees = sees & ~dead[None, :]
    any_key = sees.any(1)
    used = sees.any(0)
    for h in range(H):
        qd, kd, vd = q[:, h].double(), k[:, h // (H // G)].double(), v[:, h // (H // G)].double()
        kd = torch.where(used[:, None], kd, 0.0)
        vd = torch.where(used[:, None], vd, 0.0)
        s = scale * (qd @ kd.t())
        s = s.masked_fill(~sees, -float("inf"))
        p = torch.softmax(torch.where(any_key[:, None], s, 0.0), dim=1)
        p = torch.where(any_key[:, None] & sees, p, 0.0)
        o, w = p @ vd, p @ vd.abs()
        d = (D + 8) * 2.0 ** -23 * scale * (qd.abs() @ kd.abs().t()).amax(1, keepdim=True)
        out[:, h] = o
        tol[:, h] = 2.0 ** -8 * o.abs() + w * (2 * d + 2.0 ** -8 + 2 * m * 2.0 ** -23 + 2.0 ** -12)
    return out, tol


def check(out, ref, tol, what):
    err = (out.double() - ref).abs()
    assert bool(torch.isfinite(out.float()).all()), "%s: not finite" % what
    assert bool((err <= tol + 1e-30).all()), "%s: worst %.3g of the bound" % (
        what, float((err / (tol + 1e-30)).max()))


def normal(seed, *shape, gain=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (gain * torch.randn(shape, generator=g, device=DEV)).to(BF)


# ------------------------------------------------------------------ packed

PACKED = [
    # H, G, D, lens
    (1, 1, 128, [1]), (1, 1, 64, [1]), (2, 1, 64, [63]), (3, 3, 128, [64]), (4, 1, 128, [65]),
    (5, 5, 64, [2, 1, 3]), (6, 2, 128, [127, 0, 128, 129]), (8, 8, 64, [300, 77, 1]),
    (7, 1, 128, [100, 1, 257]), (12, 4, 64, [511, 0, 0, 513]), (16, 1, 128, [33, 34]),
    (64, 1, 64, [9, 40]), (24, 8, 128, [640, 1000]), (10, 2, 64, [1500]), (4, 2, 128, [3001]),
    (3, 1, 128, [200, 1] * 40), (2, 2, 64, [5] * 130 + [700]), (8, 2, 128, [0, 0, 2048, 0]),
    # many pairs of a row and a key: tiles of 256 rows
    (32, 8, 128, [3000]), (32, 4, 64, [2999]), (40, 8, 128, [2500, 0, 1900, 900]), (48, 48, 64, [285] * 70 + [3]),
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("H,G,D,lens", PACKED)
def test_packed_attention(H, G, D, lens, causal):
    T = sum(lens)
    q, k, v = normal(1, T, H, D, gain=1.5), normal(2, T, G, D), normal(3, T, G, D)
    at = starts_of(lens)
    out = bdt.packed_attention(q, k, v, ints(at), causal=causal)
    assert out.shape == (T, H, D)
    for a, b in zip(at[:-1], at[1:]):
        ref, tol = sequence_64(q[a:b], k[a:b], v[a:b], D ** -0.5, causal)
        check(out[a:b], ref, tol, "rows %d .. %d" % (a, b))
    assert torch.equal(bdt.packed_attention(q, k, v, ints(at), causal=causal), out)


@pytest.mark.parametrize("B", [65, 4096, 4097, 9000])
def test_many_sequences(B):
    """Against the same rows as equal sequences of one batched form."""
    H, G, D, n = 3, 1, 64, 5
    T = B * n
    q, k, v = normal(1, T, H, D), normal(2, T, G, D), normal(3, T, G, D)
    out = bdt.packed_attention(q, k, v, ints([n * i for i in range(B + 1)]))
    x, y, z = (t.view(B, n, -1, D).double().transpose(1, 2) for t in (q, k, v))
    s = D ** -0.5 * (x @ y.transpose(-1, -2).contiguous())
    s = s.masked_fill(torch.ones(n, n, dtype=torch.bool, device=DEV).triu(1), -float("inf"))
    p = torch.softmax(s, -1)
    ref, w = p @ z, p @ z.abs()
    d = (D + 8) * 2.0 ** -23 * D ** -0.5 * (x.abs() @ y.abs().transpose(-1, -2).contiguous()).amax(-1, keepdim=True)
    tol = 2.0 ** -8 * ref.abs() + w * (2 * d + 2.0 ** -8 + 2 * n * 2.0 ** -23 + 2.0 ** -12)
    check(out, ref.transpose(1, 2).reshape(T, H, D), tol.transpose(1, 2).reshape(T, H, D), "%d sequences" % B)
    # every second one empty, its rows left to its neighbour
    at = [n * (i - i % 2) for i in range(B)] + [T]
    got = bdt.packed_attention(q, k, v, ints(at), causal=False)
    for b in (0, 1, 2, 63, 64, B // 2, B - 2, B - 1):
        r = slice(at[b], at[b + 1])
        check(got[r], *sequence_64(q[r], k[r], v[r], D ** -0.5, False), "sequence %d of %d" % (b, B))


@pytest.mark.parametrize("H,G,D,lens,keys", [
    (2, 1, 128, [3, 1, 70], [500, 0, 70]), (4, 4, 64, [1], [4000]), (6, 2, 128, [130, 5], [64, 3000]),
    (8, 2, 128, [1, 1, 1, 200], [1, 0, 2000, 199]), (2, 2, 64, [300], [10]),
    (12, 12, 128, [1560, 77], [400, 333]),
])
@pytest.mark.parametrize("causal", [True, False])
def test_keys_of_their_own(H, G, D, lens, keys, causal):
    """Fewer keys than rows: with causal the first rows see none."""
    T, Tk = sum(lens), sum(keys)
    q, k, v = normal(4, T, H, D), normal(5, Tk, G, D), normal(6, Tk, G, D)
    qa, ka = starts_of(lens), starts_of(keys)
    out = bdt.packed_attention(q, k, v, ints(qa), ints(ka), causal=causal, scale=0.2)
    for i in range(len(lens)):
        x, y = slice(qa[i], qa[i + 1]), slice(ka[i], ka[i + 1])
        ref, tol = sequence_64(q[x], k[y], v[y], 0.2, causal)
        check(out[x], ref, tol, "sequence %d" % i)
        if causal and lens[i] > keys[i]:
            assert bool((out[x][:lens[i] - keys[i]] == 0).all())


@pytest.mark.parametrize("D", [64, 128])
def test_parts_of_a_projection(D):
    """q, k and v as columns of one projection, and rows behind the last sequence."""
    H, G, lens = 6, 2, [70, 0, 333]
    T = sum(lens) + 9
    qkv = normal(7, T, (H + 2 * G) * D)
    q, k, v = (x.view(T, -1, D) for x in qkv.split([H * D, G * D, G * D], dim=1))
    assert not q.is_contiguous()
    buf = torch.full((T, H, D), -777.0, dtype=BF, device=DEV)
    out = bdt.packed_attention(q, k, v, ints(starts_of(lens)), out=buf)
    assert out is buf and bool((buf[-9:] == -777).all())
    want = bdt.packed_attention(q.contiguous(), k.contiguous(), v.contiguous(), ints(starts_of(lens)))
    assert torch.equal(out[:-9], want[:-9])
    bits = bdt.packed_attention(q.view(torch.int16), k.view(torch.int16), v, ints(starts_of(lens)))
    assert torch.equal(bits[:-9], want[:-9])


# ------------------------------------------------------------------ paged

def paged_inputs(H, G, D, page, new, lens, seed, spare=3, gain=1.0):
    """(q, k_cache, v_cache, tables, dense k, dense v): pages in a mixed order; what no request
    holds is NaN or infinite."""
    T, each = sum(new), [-(-n // page) for n in lens]
    pages, width = sum(each) + spare, max(each + [0]) + 2
    q = normal(seed, T, H, D, gain=gain)
    kc = torch.full((pages, G, page, D), float("nan"), dtype=BF, device=DEV)
    vc = torch.full((pages, G, page, D), float("inf"), dtype=BF, device=DEV)
    vc[..., ::2] = float("nan")
    order = np.random.default_rng(seed).permutation(pages)
    tables = np.full((len(new), width), 7 * pages + 11, np.int64)
    tables[:, 1::2] = -5
    ks, vs, at = [], [], 0
    for b, n in enumerate(lens):
        k, v = normal(seed + 10 + b, n, G, D), normal(seed + 1000 + b, n, G, D)
        ks.append(k)
        vs.append(v)
        for i in range(each[b]):
            p = int(order[at])
            at += 1
            tables[b, i] = p
            part = slice(i * page, min((i + 1) * page, n))
            kc[p, :, :part.stop - part.start] = k[part].transpose(0, 1)
            vc[p, :, :part.stop - part.start] = v[part].transpose(0, 1)
    return q, kc, vc, ints(tables.astype(np.int32).tolist()).view(len(new), width), ks, vs


PAGED = [
    # H, G, D, page, new, lens
    (1, 1, 128, 16, [1], [1]), (1, 1, 64, 16, [1], [17]), (8, 2, 128, 64, [1], [5000]),
    (32, 8, 128, 16, [1] * 9, [9, 1, 16, 17, 333, 64, 65, 4097, 128]), (4, 4, 64, 32, [1, 1], [0, 100]),
    (6, 1, 128, 128, [1, 0, 2, 5], [300, 50, 700, 5]), (16, 1, 64, 256, [1, 1, 1], [2000, 256, 257]),
    (12, 12, 128, 64, [3, 1], [1000, 999]), (28, 4, 64, 32, [1, 1, 130, 1], [90, 300, 800, 31]),
    (4, 2, 128, 16, [64], [64]), (8, 1, 128, 64, [40, 17], [3000, 17]), (2, 2, 128, 256, [700], [1500]),
    (5, 5, 64, 16, [129], [3000]), (64, 1, 128, 16, [1, 3], [700, 4]), (3, 1, 128, 64, [1] * 70, list(range(1, 140, 2))),
    (8, 8, 128, 64, [5, 5], [3, 5]), (24, 24, 64, 64, [1], [20000]), (10, 2, 128, 32, [16, 7], [2222, 4444]),
    (16, 2, 128, 128, [2, 4, 1], [9000, 31, 12000]),
    # many rows: tiles of 256 rows, and requests of few rows beside them
    (32, 8, 128, 64, [1] * 20 + [600] + [2, 8, 9, 0], list(range(1, 4000, 200)) + [1700, 900, 8, 9, 77]),
    (28, 4, 64, 32, [4, 1200, 1, 5], [3333, 1200, 5000, 1]), (24, 24, 128, 256, [32, 800, 33], [1000, 801, 600]),
    (20, 1, 64, 16, [1, 1, 2, 1700], [7000, 300, 90, 1750]),
    # a tile for each of twice the workers
    (8, 8, 128, 32, [1] * 130, list(range(1, 651, 5))), (12, 6, 64, 16, [1, 2, 0, 1, 1] * 69, [7, 300, 20, 1, 99] * 69),
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("H,G,D,page,new,lens", PAGED)
def test_paged_attention(H, G, D, page, new, lens, causal):
    q, kc, vc, tables, ks, vs = paged_inputs(H, G, D, page, new, lens, 20)
    at, kv = starts_of(new), ints(lens)
    outs = [bdt.paged_attention(q, kc, vc, tables, ints(at), kv, max_new=most, causal=causal)
            for most in (max(new), None, 1)]
    for out in outs:
        for b in range(len(new)):
            x = slice(at[b], at[b + 1])
            ref, tol = sequence_64(q[x], ks[b], vs[b], D ** -0.5, causal)
            check(out[x], ref, tol, "request %d" % b)
    assert torch.equal(bdt.paged_attention(q, kc, vc, tables, ints(at), kv, max_new=max(new),
                                           causal=causal), outs[0])


@pytest.mark.parametrize("H,G,new,lens", [(8, 2, [1, 1], [900, 130]), (4, 4, [70, 1], [900, 130]),
                                          (16, 2, [3, 2], [900, 130])])
@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("D", [64, 128])
def test_pages_outside_the_cache_hold_no_keys(D, page, H, G, new, lens):
    q, kc, vc, tables, ks, vs = paged_inputs(H, G, D, page, new, lens, 3)
    host = tables.cpu()
    dead = [torch.zeros(n, dtype=torch.bool, device=DEV) for n in lens]
    for b, i, entry in ((0, 1, -1), (0, 2, kc.shape[0]), (1, 0, 2 ** 31 - 1), (0, 3, -2 ** 31)):
        if i * page < lens[b]:
            host[b, i] = entry
            dead[b][i * page:(i + 1) * page] = True
    at = starts_of(new)
    out = bdt.paged_attention(q, kc, vc, host.to(DEV), ints(at), ints(lens), max_new=max(new))
    for b in range(2):
        x = slice(at[b], at[b + 1])
        ref, tol = sequence_64(q[x], ks[b], vs[b], D ** -0.5, True, dead[b])
        check(out[x], ref, tol, "request %d" % b)
    host.fill_(-1)
    out = bdt.paged_attention(q, kc, vc, host.to(DEV), ints(at), ints(lens), max_new=max(new))
    assert bool((out == 0).all())
    none = bdt.paged_attention(q, kc[:0], vc[:0], tables, ints(at), ints(lens), max_new=max(new))
    assert bool((none == 0).all())


@pytest.mark.parametrize("D,chunk", [(64, 3), (128, 1100)])
def test_many_long_requests_in_tiles(D, chunk):
    """So many that a workgroup has thousands of keys of one request of few rows; a page is missing."""
    H, page, n = 16, 64, 9000
    new, lens = [1] * 40 + [chunk], [n - 7 * b for b in range(40)] + [chunk]
    q, kc, vc, tables, ks, vs = paged_inputs(H, H, D, page, new, lens, 8)
    tables[1, 130] = -1
    dead = torch.zeros(lens[1], dtype=torch.bool, device=DEV)
    dead[130 * page:131 * page] = True
    at = starts_of(new)
    for most in (None, 1):
        out = bdt.paged_attention(q, kc, vc, tables, ints(at), ints(lens), max_new=most)
        for b in (0, 1, 2, 17, 39, 40):
            x = slice(at[b], at[b + 1])
            ref, tol = sequence_64(q[x], ks[b], vs[b], D ** -0.5, True, dead if b == 1 else None)
            check(out[x], ref, tol, "request %d" % b)


def test_lengths_past_the_table_and_starts_out_of_order():
    """Lengths are clamped to the table's width; starts are clamped, and a sequence that ends
    before it starts has no rows; rows of no sequence stay."""
    H, G, D, page = 4, 2, 128, 16
    q, kc, vc, tables, ks, vs = paged_inputs(H, G, D, page, [2, 3], [48, 48], 5)
    full = tables[:, :3].contiguous()
    want = bdt.paged_attention(q, kc, vc, full, ints([0, 2, 5]), ints([48, 48]))
    got = bdt.paged_attention(q, kc, vc, full, ints([0, 2, 5]), ints([49, 2 ** 31 - 1]))
    assert torch.equal(got, want)
    buf = torch.full_like(q, -777.0)
    bdt.paged_attention(q, kc, vc, full, ints([-7, 2, 1]), ints([48, -3]), out=buf)
    assert torch.equal(buf[:2], want[:2]) and bool((buf[2:] == -777).all())
    buf.fill_(-777.0)
    bdt.paged_attention(q, kc, vc, full, ints([2, 5, 2 ** 31 - 1]), ints([0, 48]), out=buf)
    assert bool((buf[:2] == -777).all()) and bool((buf[2:] == 0).all())


@pytest.mark.parametrize("seed", range(16))
def test_drawn_shapes(seed):
    """Heads, lengths, pages and strides at random, over the cache and packed."""
    rng = np.random.default_rng(seed)
    G = int(rng.choice([1, 2, 3, 5, 8]))
    H, D = G * int(rng.choice([1, 2, 3, 4, 7, 16])), int(rng.choice([64, 128]))
    B, page = int(rng.integers(1, 90 if seed % 4 == 0 else 8)), int(rng.choice([16, 32, 64, 128, 256]))
    causal, most = bool(rng.integers(2)), int(rng.choice([1, 3, 40, 300]))
    new = rng.integers(0 if B > 1 else 1, most + 1, B).tolist()
    if sum(new) == 0:
        new[0] = 1
    lens = [int(n + rng.integers(0, 1 + int(rng.choice([1, 100, 2000])))) for n in new]
    q, kc, vc, tables, ks, vs = paged_inputs(H, G, D, page, new, lens, 100 + seed)
    at = starts_of(new)
    outs = [bdt.paged_attention(q, kc, vc, tables, ints(at), ints(lens), max_new=m, causal=causal)
            for m in (max(max(new), 1), 4000)]
    wide = normal(seed, sum(new), H * D + 8 * int(rng.integers(1, 5)))       # rows that lie apart
    wide[:, :H * D] = q.view(sum(new), H * D)
    k, v = torch.cat(ks), torch.cat(vs)
    outs.append(bdt.packed_attention(wide[:, :H * D].unflatten(1, (H, D)), k, v, ints(at), ints(starts_of(lens)),
                                     causal=causal))
    for b in range(B):
        x = slice(at[b], at[b + 1])
        ref, tol = sequence_64(q[x], ks[b], vs[b], D ** -0.5, causal)
        for out, what in zip(outs, ("for its most", "in tiles", "packed")):
            check(out[x], ref, tol, "request %d, %s" % (b, what))


# ------------------------------------------------------------------ values

@pytest.mark.parametrize("gain", [0.0, 40.0, 4000.0])
@pytest.mark.parametrize("new,lens", [([1, 1], [3000, 70]), ([300, 2], [2000, 40])])
def test_extreme_scores(gain, new, lens):
    H, G, D = 4, 2, 128
    q, kc, vc, tables, ks, vs = paged_inputs(H, G, D, 64, new, lens, 9, gain=gain)
    at = starts_of(new)
    out = bdt.paged_attention(q, kc, vc, tables, ints(at), ints(lens), max_new=max(new))
    for b in range(2):
        x = slice(at[b], at[b + 1])
        ref, tol = sequence_64(q[x], ks[b], vs[b], D ** -0.5, True)
        check(out[x], ref, tol, "gain %g" % gain)


@pytest.mark.parametrize("H,G,D,lens", [(4, 1, 128, [200, 300]), (2, 2, 64, [130, 700]), (8, 2, 128, [10, 20]),
                                        (1, 1, 128, [3000])])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_later_keys_that_are_not_finite_stay_out_of_earlier_rows(H, G, D, lens, bad):
    T, at = sum(lens), starts_of(lens)
    q, k, v = normal(1, T, H, D), normal(2, T, G, D), normal(3, T, G, D)
    clean = bdt.packed_attention(q, k, v, ints(at))
    n = at[-1] - 5                                   # a late key of the last sequence
    kb, vb = k.clone(), v.clone()
    kb[n], vb[n, :, 3] = float("nan"), bad
    out = bdt.packed_attention(q, kb, vb, ints(at))
    assert torch.equal(out[:n], clean[:n])
    assert bool(out[n:].isnan().all())
    out = bdt.packed_attention(q, k, vb, ints(at))
    assert torch.equal(out[:n], clean[:n])
    other = [d for d in range(D) if d != 3]
    assert torch.equal(out[n:][..., other], clean[n:][..., other])
    assert not bool(torch.isfinite(out[n:, :, 3]).any())


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("H,G,D,new,lens", [(8, 2, 128, [5, 200, 8], [1000, 300, 40]), (8, 2, 64, [5, 200, 8], [1000, 300, 40]),
                                            (32, 8, 128, [3, 600, 8], [5000, 700, 9]), (12, 2, 64, [2, 5], [3000, 5])])
def test_later_values_of_a_cache_stay_out_of_earlier_rows(H, G, D, new, lens, bad):
    """The last key of each request, which only its last token sees."""
    page = 32
    q, kc, vc, tables, ks, vs = paged_inputs(H, G, D, page, new, lens, 4)
    at, kv = starts_of(new), ints(lens)
    clean = bdt.paged_attention(q, kc, vc, tables, ints(at), kv, max_new=max(new))
    for b, n in enumerate(lens):
        vc[tables[b, (n - 1) // page], :, (n - 1) % page, 3] = bad
    out = bdt.paged_attention(q, kc, vc, tables, ints(at), kv, max_new=max(new))
    last = torch.zeros(sum(new), dtype=torch.bool, device=DEV)
    last[[x - 1 for x in at[1:]]] = True
    assert torch.equal(out[~last], clean[~last])
    assert not bool(torch.isfinite(out[last][..., 3]).any())
    other = [d for d in range(D) if d != 3]
    assert torch.equal(out[last][..., other], clean[last][..., other])


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("new,lens", [([1, 1], [4000, 70]), ([200, 2], [2000, 40])])
def test_a_query_that_is_not_finite(bad, new, lens):
    H, G, D = 4, 2, 128
    q, kc, vc, tables, ks, vs = paged_inputs(H, G, D, 64, new, lens, 9)
    args = (kc, vc, tables, ints(starts_of(new)), ints(lens))
    clean = bdt.paged_attention(q, *args, max_new=max(new))
    q[0, 1, 77] = bad
    out = bdt.paged_attention(q, *args, max_new=max(new))
    assert bool(out[0, 1].isnan().all())
    out[0, 1] = clean[0, 1]
    assert torch.equal(out, clean)


@pytest.mark.parametrize("new", [[3, 1], [40, 1]])
def test_a_query_that_is_not_finite_and_sees_no_key(new):
    q, kc, vc, tables, _, _ = paged_inputs(4, 2, 64, 16, new, [2, 1], 3)
    q[0] = float("nan")
    out = bdt.paged_attention(q, kc, vc, tables, ints(starts_of(new)), ints([2, 1]), max_new=max(new))
    assert bool((out[0] == 0).all()) and bool(torch.isfinite(out.float()).all())


@pytest.mark.parametrize("new", [1, 70])
def test_a_key_that_is_infinite(new):
    """No weight where the score is minus infinity, NaN elsewhere."""
    n, D = 2000, 64
    q, kc, vc, tables, ks, vs = paged_inputs(1, 1, D, 16, [new], [n], 3)
    q[:, 0, 0] = q[:, 0, 0].abs() + 0.1
    kc[tables[0, 3], 0, 5, 0] = -float("inf")                  # key 53
    dead = torch.zeros(n, dtype=torch.bool, device=DEV)
    dead[53] = True
    args = (kc, vc, tables, ints([0, new]), ints([n]))
    out = bdt.paged_attention(q, *args, max_new=new)
    ref, tol = sequence_64(q, ks[0], vs[0], D ** -0.5, True, dead)
    check(out, ref, tol, "minus infinity")
    kc[tables[0, 3], 0, 5, 0] = float("inf")
    assert bool(bdt.paged_attention(q, *args, max_new=new).isnan().all())


def test_outputs_and_workspace_stay_inside():
    for H, G, D, new, lens in ((4, 2, 128, [1, 1], [3000, 500]), (6, 2, 64, [150, 3], [1000, 40])):
        q, kc, vc, tables, _, _ = paged_inputs(H, G, D, 64, new, lens, 2)
        T, at = sum(new), ints(starts_of(new))
        s = bdt.PagedShape(T, kc.shape[0], H * D, len(new), H, G, D, 64, tables.shape[1], max(new), 1)
        need = bdt.svdq_paged_attention_workspace_bytes(s)
        n = q.numel()
        buf = torch.full((n + 512,), -777.0, dtype=BF, device=DEV)
        ws = torch.full((need + 512,), 0xFF, dtype=torch.uint8, device=DEV)
        bdt.svdq_paged_attention(q, kc, vc, tables, at, ints(lens), s, D ** -0.5, buf[256:256 + n],
                                 ws[256:], need)
        assert bool((buf[:256] == -777).all()) and bool((buf[256 + n:] == -777).all())
        assert bool((ws[:256] == 0xFF).all()) and bool((ws[256 + need:] == 0xFF).all())
        out = bdt.paged_attention(q, kc, vc, tables, at, ints(lens), max_new=max(new))
        assert torch.equal(buf[256:256 + n].view_as(out), out)


@pytest.mark.parametrize("new", [[1, 1, 1], [90, 1, 40]])
def test_in_a_graph_and_on_two_streams(new):
    H, G, D, page = 8, 2, 128, 32
    lens = [2000, 300, 777]
    sets = [paged_inputs(H, G, D, page, new, lens, seed)[:4] for seed in (1, 2)]
    at, kv = ints(starts_of(new)), ints(lens)

    def call(q, kc, vc, t, kv=kv):
        return bdt.paged_attention(q, kc, vc, t, at, kv, max_new=max(new))
    want = [call(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        got = []
        for st, s in zip(streams, sets):
            with torch.cuda.stream(st):
                got.append(call(*s))
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    mine = [x.clone() for x in sets[0]]
    length = kv.clone()
    with torch.cuda.stream(streams[0]):
        call(*mine, kv=length)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(*mine, kv=length)
    for it in range(5):
        for dst, src in zip(mine, sets[it % 2]):
            dst.copy_(src)
        length.copy_(kv if it < 3 else kv // 3)                # lengths read at replay
        graph.replay()
        torch.cuda.synchronize()
        eager = call(*mine, kv=length)
        assert torch.equal(out, eager), "replay %d" % it
        if it < 3:
            assert torch.equal(out, want[it % 2])


def test_packed_in_a_graph_and_on_two_streams():
    """Two graphs of packed calls, replayed on two streams at once."""
    sets = [(normal(s, 700, 6, 64), normal(s + 1, 700, 2, 64), normal(s + 2, 700, 2, 64)) for s in (1, 5)]
    at = ints([0, 600, 600, 690])
    want = [bdt.packed_attention(*s, at) for s in sets]
    torch.cuda.synchronize()
    streams, graphs, outs = [torch.cuda.Stream(), torch.cuda.Stream()], [], []
    for s in sets:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(bdt.packed_attention(*s, at, out=torch.full_like(s[0], -3.0)))
    for _ in range(4):
        for st, g in zip(streams, graphs):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for s, o, w in zip(sets, outs, want):
            assert torch.equal(o[:690], w[:690]) and bool((o[690:] == -3).all())
            assert torch.equal(bdt.packed_attention(*s, at)[:690], w[:690])
            o[:690].fill_(0)


def test_no_columns():
    x = torch.empty(3, 4, 0, dtype=BF, device=DEV)
    with pytest.raises(RuntimeError, match="head_dim"):
        bdt.packed_attention(x, x, x, ints([0, 3]))


def test_offsets_past_32_bits():
    """A cache of more than 2^31 elements; the request's pages are its last ones."""
    G, page, D, n = 8, 256, 128, 700
    pages = 8300
    kc = torch.zeros(pages, G, page, D, dtype=BF, device=DEV)
    assert kc.numel() > 1 << 31
    vc = torch.zeros_like(kc)
    k, v = normal(1, n, G, D), normal(2, n, G, D)
    table = [pages - 1, pages - 3, pages - 2]
    for i, p in enumerate(table):
        part = slice(i * page, min((i + 1) * page, n))
        kc[p, :, :part.stop - part.start] = k[part].transpose(0, 1)
        vc[p, :, :part.stop - part.start] = v[part].transpose(0, 1)
    for m in (1, 60):
        q = normal(3, m, 2 * G, D)
        out = bdt.paged_attention(q, kc, vc, ints([table]), ints([0, m]), ints([n]), max_new=m)
        ref, tol = sequence_64(q, k, v, D ** -0.5, True)
        check(out, ref, tol, "%d rows" % m)


def test_empty():
    q = torch.empty(0, 4, 64, dtype=BF, device=DEV)
    k = torch.empty(0, 2, 64, dtype=BF, device=DEV)
    assert bdt.packed_attention(q, k, k, ints([0])).shape == (0, 4, 64)
    assert bdt.packed_attention(q, k, k, ints([0, 0])).shape == (0, 4, 64)
    q = normal(1, 3, 4, 64)
    out = bdt.packed_attention(q, k, k, ints([0, 3]), ints([0, 0]), causal=False)
    assert bool((out == 0).all())
    buf = torch.full_like(q, 5.0)
    assert bool((bdt.packed_attention(q, q, q, ints([0]), out=buf) == 5).all())

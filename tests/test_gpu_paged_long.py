"""Attention over many keys with inputs on which one lost, doubled or unmasked block, page or key
shows (tests/long_keys.py; tests/test_long_keys.py plants the mistakes): packed, over a cache with
few new tokens, with many, and with both beside each other."""
import pytest
import torch

import bit_diffusion_transformer_amd as bdt
from tests import long_keys as lk
from tests.helpers import DEV

pytestmark = pytest.mark.gpu

# H, G, D, page (None: packed), new tokens, keys of each sequence
CASES = [
    (24, 24, 64, 64, [1], [20000]), (32, 8, 128, 64, [1], [65537]), (8, 2, 64, 32, [1], [40000]),
    (16, 2, 128, 128, [2, 4, 1], [9000, 31, 12000]), (8, 2, 128, 16, [1] * 5, [5000, 16384, 64, 8191, 4097]),
    (12, 6, 64, 16, [3, 1, 5], [7000, 16384, 999]),
    (32, 8, 128, 64, [1] * 5 + [600], [9000, 64, 65, 4097, 3000, 1700]), (28, 4, 64, 32, [4, 1200, 1], [3333, 2048, 16384]),
    (2, 2, 128, 256, [700], [3000]), (5, 5, 64, 16, [129], [16384]), (16, 16, 64, 64, [1] * 12 + [3], [9000 - 7 * b for b in range(12)] + [4096]),
    (4, 2, 128, None, [3001], [3001]), (8, 2, 128, None, [5000, 1, 700], [5000, 1, 700]), (6, 2, 64, None, [4096, 333], [4096, 333]),
    (32, 8, 128, None, [3000], [3000]), (4, 1, 64, None, [1, 130], [16384, 9000]),
]
CASES_IDS = ["%s-%d-%d-%d-%s" % ("packed" if c[3] is None else "paged%d" % c[3], c[0], c[1], c[2], max(c[5])) for c in CASES]
cases = pytest.mark.parametrize("H,G,D,page,new,lens", CASES, ids=CASES_IDS)


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def starts(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return at


def outputs(qs, ks, vs, page, new, lens, causal, scale, dead=None):
    """The outputs of every way to call it, one list of the sequences' rows each.  dead: (request,
    entry of its table) pairs whose page is taken away."""
    q, at = torch.cat(qs), starts(new)
    if page is None:
        outs = [bdt.packed_attention(q, torch.cat(ks), torch.cat(vs), ints(at), ints(starts(lens)), causal=causal, scale=scale)]
    else:
        kc, vc, tables = lk.in_pages(ks, vs, page, 7)
        for b, i in dead or ():
            tables[b, i] = -1 if b % 2 else kc.shape[0]
        outs = [bdt.paged_attention(q, kc, vc, tables.to(DEV), ints(at), ints(lens), max_new=most, causal=causal, scale=scale)
                for most in (max(new), None, 1)]
    return [[out[a:b] for a, b in zip(at[:-1], at[1:])] for out in outs]


@pytest.mark.parametrize("causal", [True, False])
@cases
def test_random_values(H, G, D, page, new, lens, causal):
    qs = [lk.normal(10 + b, n, H, D, device=DEV) for b, n in enumerate(new)]
    ks = [lk.normal(100 + b, m, G, D, device=DEV) for b, m in enumerate(lens)]
    vs = [lk.normal(1000 + b, m, G, D, device=DEV) for b, m in enumerate(lens)]
    outs = outputs(qs, ks, vs, page, new, lens, causal, D ** -0.5)
    for b, (n, m) in enumerate(zip(new, lens)):
        if m < 1000:
            continue
        sees = lk.visible(n, m, causal, device=DEV)
        rows = sees.sum(1) >= 1000
        ref, _ = lk.exact(qs[b], ks[b], vs[b], D ** -0.5, sees)
        for out in outs:
            lk.check_rms(out[b][rows], ref[rows], "sequence %d" % b)


@pytest.mark.parametrize("causal", [True, False])
@cases
def test_counted_keys(H, G, D, page, new, lens, causal):
    made = [lk.counted(n, m, H, G, D, device=DEV) for n, m in zip(new, lens)]
    outs = outputs(*zip(*made), page, new, lens, causal, 1.0)
    for b, (n, m) in enumerate(zip(new, lens)):
        for out in outs:
            lk.check_counted(out[b], made[b][2], lk.visible(n, m, causal, device=DEV), "sequence %d" % b)


@pytest.mark.parametrize("causal", [True, False])
@cases
def test_peaks(H, G, D, page, new, lens, causal):
    """Weights that halve with each key away from one: first and last keys, ends of blocks, and the
    last key that a row sees where the peak is behind it."""
    made = []
    for n, m in zip(new, lens):
        at = [m - 1, 0, 63, 64, m // 2, m - 65, 31, 32, m // 3 // 64 * 64, m - 2, 127, 128]
        made.append(lk.peaked(n, m, H, G, D, [min(max(at[g % len(at)], 0), m - 1) for g in range(G)], device=DEV))
    outs = outputs(*zip(*made), page, new, lens, causal, lk.LN2)
    for b, (n, m) in enumerate(zip(new, lens)):
        ref, size = lk.exact(*made[b], lk.LN2, lk.visible(n, m, causal, device=DEV))
        for out in outs:
            lk.check_powers(out[b], ref, size, "sequence %d" % b)


@cases
def test_far_scores(H, G, D, page, new, lens):
    made = [lk.far(n, m, H, G, D, 30 + b, device=DEV) for b, (n, m) in enumerate(zip(new, lens))]
    outs = outputs(*zip(*made), page, new, lens, True, lk.THIRD)
    for b, (n, m) in enumerate(zip(new, lens)):
        ref, size = lk.exact(*made[b], lk.THIRD, lk.visible(n, m, True, device=DEV))
        for out in outs:
            lk.check_thirds(out[b], ref, size, "sequence %d" % b)


@pytest.mark.parametrize("H,G,D,page,new,lens", [c for c in CASES if c[3]], ids=[i for c, i in zip(CASES, CASES_IDS) if c[3]])
def test_pages_that_are_missing(H, G, D, page, new, lens):
    """Their keys would outscore all others, with values of a hundred."""
    qs = [lk.normal(10 + b, n, H, D, device=DEV) for b, n in enumerate(new)]
    ks = [lk.normal(100 + b, m, G, D, device=DEV) for b, m in enumerate(lens)]
    vs = [lk.normal(1000 + b, m, G, D, device=DEV) for b, m in enumerate(lens)]
    gone, dead = [], []
    for b, m in enumerate(lens):
        dead.append(torch.zeros(m, dtype=torch.bool, device=DEV))
        qs[b][..., 0], ks[b][..., 0] = 8.0, 0.0
        for i in {0, 3, m // page // 2, m // page - 1} if m >= 8 * page else ():
            gone.append((b, i))
            rows = slice(i * page, (i + 1) * page)
            dead[b][rows], ks[b][rows, :, 0], vs[b][rows] = True, 16.0, 100.0
    outs = outputs(qs, ks, vs, page, new, lens, True, D ** -0.5, gone)
    for b, (n, m) in enumerate(zip(new, lens)):
        if m < 1000:
            continue
        sees = lk.visible(n, m, True, dead[b], device=DEV)
        rows = sees.sum(1) >= 1000
        ref, _ = lk.exact(qs[b], ks[b], vs[b], D ** -0.5, sees)
        for out in outs:
            lk.check_rms(out[b][rows], ref[rows], "request %d" % b)

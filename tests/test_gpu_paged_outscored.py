"""A v that is not finite shows in its column of every row that sees its key, also where the
key's weight underflows to zero, wherever in a block of keys, beside a mask or not."""
import numpy as np
import pytest
import torch

import bit_diffusion_transformer_amd as bdt
from tests.helpers import DEV
from tests.test_gpu_paged import ints, normal, paged_inputs, starts_of

pytestmark = pytest.mark.gpu
BAD = [float("nan"), float("inf"), -float("inf")]


def outscored(q, k):
    """A key that every row of q gives a score below the others' by 200 and more: exp(-200) is no
    fp32 number.  (q and k get a column of their own: 16 in q, 0 in k, -256 in that key.)"""
    q[..., 0], k[..., 0] = 16.0, 0.0
    key = k[0].clone()
    key[..., 0] = -256.0
    return key


def compare(out, clean, sees):
    """Rows that see the key: column 3 is not finite; all else is as without the bad value."""
    other = [d for d in range(out.shape[-1]) if d != 3]
    assert torch.equal(out[~sees], clean[~sees])
    assert torch.equal(out[..., other], clean[..., other])
    assert not bool(torch.isfinite(out[sees][..., 3]).any())


@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("H,G,D,n", [(4, 1, 128, 300), (2, 2, 64, 130), (32, 8, 128, 2900), (8, 2, 64, 3)])
def test_packed(H, G, D, n, causal, bad):
    q, k, v = normal(1, n, H, D), normal(2, n, G, D), normal(3, n, G, D)
    key, scale = outscored(q, k), 0.125
    rows = torch.arange(n, device=DEV)
    for j in {0, 1, n // 2, n - 2, n - 1}:
        kb, vb = k.clone(), v.clone()
        kb[j] = key
        clean = bdt.packed_attention(q, kb, v, ints([0, n]), causal=causal, scale=scale)
        vb[j, :, 3] = bad
        out = bdt.packed_attention(q, kb, vb, ints([0, n]), causal=causal, scale=scale)
        sees = rows >= j if causal else rows >= 0
        if causal and j == 0:
            sees = rows > 0                # (row 0 sees that key alone: its weight is one)
            assert not bool(torch.isfinite(out[0, :, 3]).any())
            out[0], clean[0] = 0, 0
        compare(out, clean, sees)


@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("missing", [False, True])
@pytest.mark.parametrize("H,G,D,new,lens", [
    (8, 2, 128, [1], [300]), (8, 2, 64, [1, 3], [777, 1000]), (16, 2, 128, [4, 1], [500, 3001]),   # few rows
    (32, 8, 128, [3, 600, 8], [1000, 700, 333]), (28, 4, 64, [2, 1200, 4], [900, 1500, 2222]),      # and beside many
    (6, 2, 128, [200, 70], [300, 1000])])
def test_paged(H, G, D, new, lens, missing, bad):
    """missing: a page of another 16 keys in the same block of 32 or 64 is outside the cache."""
    page, scale = 16, 0.125
    q, kc, vc, tables, ks, vs = paged_inputs(H, G, D, page, new, lens, 6)
    q[..., 0], kc[..., 0] = 16.0, 0.0
    at, kv = starts_of(new), ints(lens)
    for back in (1, 2, 40, 200, min(lens) - 2):            # the key's place from each request's end
        kb, vb, tb = kc.clone(), vc.clone(), tables.clone()
        sees = torch.zeros(sum(new), dtype=torch.bool, device=DEV)
        for b, n in enumerate(lens):
            j = n - back
            p = int(tables[b, j // page])
            kb[p, :, j % page, 0] = -256.0
            if missing:
                tb[b, j // page ^ 1] = -1
            rows = torch.arange(new[b], device=DEV)
            sees[at[b]:at[b + 1]] = rows + n - new[b] >= j
            vb[p, :, j % page, 3] = 1.0
        args = (tb, ints(at), kv)
        clean = bdt.paged_attention(q, kb, vb, *args, max_new=max(new), scale=scale)
        for b, n in enumerate(lens):
            vb[int(tables[b, (n - back) // page]), :, (n - back) % page, 3] = bad
        out = bdt.paged_attention(q, kb, vb, *args, max_new=max(new), scale=scale)
        compare(out, clean, sees)


@pytest.mark.parametrize("seed", range(12))
def test_drawn_values_show_where_their_keys_are_seen(seed):
    """Some values of some keys are not finite, and most weights are zero: a column of a row is finite
    where the row sees none of them, and nowhere else."""
    rng = np.random.default_rng(seed)
    G = int(rng.choice([1, 2, 4]))
    H, D, page = G * int(rng.choice([1, 2, 4, 8])), int(rng.choice([64, 128])), int(rng.choice([16, 32, 64]))
    causal, B, most = bool(rng.integers(2)), int(rng.integers(1, 6)), int(rng.choice([1, 4, 200, 900]))
    new = rng.integers(1, most + 1, B).tolist()
    lens = [int(n + rng.integers(0, 1 + int(rng.choice([3, 100, 1500])))) for n in new]
    q, kc, vc, tables, ks, vs = paged_inputs(H, G, D, page, new, lens, 50 + seed, gain=40.0)
    odd = []
    for b, n in enumerate(lens):
        odd.append(torch.zeros(n, G, D, dtype=torch.bool, device=DEV))
        for _ in range(1 + n // 200):
            j, g, d = int(rng.integers(n)), int(rng.integers(G)), int(rng.integers(D))
            vs[b][j, g, d] = BAD[int(rng.integers(3))]
            vc[tables[b, j // page], g, j % page, d] = vs[b][j, g, d]
            odd[b][j, g, d] = True
    at, kv = starts_of(new), ints(lens)
    outs = [bdt.paged_attention(q, kc, vc, tables, ints(at), kv, max_new=m, causal=causal) for m in (max(new), None, 1)]
    outs.append(bdt.packed_attention(q, torch.cat(ks), torch.cat(vs), ints(at), ints(starts_of(lens)), causal=causal))
    for b, (n, m) in enumerate(zip(new, lens)):
        key, row = torch.arange(m, device=DEV), torch.arange(n, device=DEV)
        sees = key[None, :] <= row[:, None] + (m - n) if causal else torch.ones(n, m, dtype=torch.bool, device=DEV)
        want = torch.einsum("nm,mgd->ngd", sees.float(), odd[b].float()) > 0
        want = want.repeat_interleave(H // G, 1)
        for out in outs:
            assert torch.equal(~torch.isfinite(out[at[b]:at[b + 1]]), want), "request %d" % b

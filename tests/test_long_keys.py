"""The checks of tests/long_keys.py against a model of the kernels on the CPU: blocks of keys with
their own maxima, weights rounded to bf16, parts joined by their maxima.  The model passes every
check; each mistake planted in it (a block, a key or a page lost, doubled or unmasked, a join or an
offset that is wrong, zeros) fails the check that is meant for it."""
import math

import pytest
import torch

from tests import long_keys as lk

BF = torch.bfloat16


def model(q, k, v, scale, sees, counts=None, blind_join=False, near_only=False):
    """Attention in parts of 64 keys.  counts [m]: how often each key is taken (1).  Mistakes:
    blind_join (every part weighs as if it had the largest maximum), near_only (the offset of an
    exponent is rounded however large it is)."""
    n, H, D = q.shape
    m, G = k.shape[:2]
    c = torch.tensor(scale, dtype=torch.float32) * 1.4426950408889634
    out = torch.zeros(n, H, D, dtype=BF)
    more = -m % 64
    counts = torch.nn.functional.pad(torch.ones(m) if counts is None else counts, (0, more)).view(-1, 1, 64)
    for h in range(H):
        s = q[:, h].float() @ k[:, h // (H // G)].float().t()
        s = torch.nn.functional.pad(s.masked_fill(~sees, -math.inf), (0, more), value=-math.inf)
        x = s.view(n, -1, 64).transpose(0, 1)                              # [parts, n, 64]
        top = x.amax(2, keepdim=True)
        off = (top * c).float()
        near = (x.double() * c.double() - off.double()).float()
        e = near if near_only else torch.where(off.abs() > 1024, ((x - top) * c).float(), near)
        p = torch.where(x > -math.inf, torch.exp2(e), 0.0).to(BF).float() * counts
        l = p.sum(2, keepdim=True)
        o = p @ torch.nn.functional.pad(v[:, h // (H // G)].float(), (0, 0, 0, more)).view(-1, 64, D)
        f = torch.ones_like(l) if blind_join else torch.exp2((top - top.amax(0)) * c)
        f = torch.where(l > 0, f, 0.0)
        acc, total = (o * f).sum(0), (l * f).sum(0)
        out[:, h] = torch.where(total > 0, acc / total.clamp(min=1e-30), 0.0).to(BF)
    return out


def taken(m, keys, times):
    c = torch.ones(m)
    c[keys] = times
    return c


LOST = [(slice(0, 64), 0), (slice(64 * 100, 64 * 101), 0), (slice(-40, None), 0), (slice(64 * 77, 64 * 78), 2),
        (slice(16 * 333, 16 * 334), 0), (slice(16 * 500, 16 * 501), 2)]


@pytest.mark.parametrize("H,G,D,m", [(2, 2, 64, 20000), (4, 1, 128, 20000), (4, 2, 128, 9000)])
def test_random_values(H, G, D, m):
    q, k, v = lk.normal(1, 2, H, D), lk.normal(2, m, G, D), lk.normal(3, m, G, D)
    sees = lk.visible(2, m, True)
    ref, _ = lk.exact(q, k, v, D ** -0.5, sees)
    lk.check_rms(model(q, k, v, D ** -0.5, sees), ref)
    for keys, times in LOST:
        with pytest.raises(AssertionError):
            lk.check_rms(model(q, k, v, D ** -0.5, sees, taken(m, keys, times)), ref)
    for mistake in (dict(blind_join=True),):
        with pytest.raises(AssertionError):
            lk.check_rms(model(q, k, v, D ** -0.5, sees, **mistake), ref)
    with pytest.raises(AssertionError):
        lk.check_rms(torch.zeros_like(q), ref)


@pytest.mark.parametrize("H,D,m", [(1, 64, 20000), (1, 128, 65537), (2, 128, 16384)])
@pytest.mark.parametrize("causal", [True, False])
def test_counted_keys(H, D, m, causal):
    q, k, v = lk.counted(3, m, H, 1, D)
    sees = lk.visible(3, m, causal)
    lk.check_counted(model(q, k, v, 1.0, sees), v, sees)
    for keys, times in LOST:
        with pytest.raises(AssertionError):
            lk.check_counted(model(q, k, v, 1.0, sees, taken(m, keys, times)), v, sees)
    if m == 16384:                                       # whole powers of two: a single key shows
        sees = lk.visible(3, m, False)
        with pytest.raises(AssertionError):
            lk.check_counted(model(q, k, v, 1.0, sees, taken(m, 5000, 0)), v, sees)


@pytest.mark.parametrize("m", [3000, 20000])
def test_peaks(m):
    peaks = [0, 63, 64, 1000, m - 1, m - 64]
    q, k, v = lk.peaked(5, m, 6, 6, 64, peaks)
    sees = lk.visible(5, m, True)
    ref, size = lk.exact(q, k, v, lk.LN2, sees)
    lk.check_powers(model(q, k, v, lk.LN2, sees), ref, size)
    for p in peaks:                                       # the key at a peak, and its block, lost or doubled
        for keys in (p, slice(p // 64 * 64, p // 64 * 64 + 64)):
            for times in (0, 2):
                if keys != p and times == 2:
                    continue                              # (a whole block that weighs all but all: no difference)
                with pytest.raises(AssertionError):
                    lk.check_powers(model(q, k, v, lk.LN2, sees, taken(m, keys, times)), ref, size)
    later = lk.visible(5, m, True).roll(1, 1)             # a mask that is off by a key
    later[:, 0] = True
    with pytest.raises(AssertionError):
        lk.check_powers(model(q, k, v, lk.LN2, later), ref, size)


@pytest.mark.parametrize("m", [150, 3000])
def test_far_scores(m):
    q, k, v = lk.far(7, m, 4, 2, 128, 3)
    sees = lk.visible(7, m, False)
    ref, size = lk.exact(q, k, v, lk.THIRD, sees)
    lk.check_thirds(model(q, k, v, lk.THIRD, sees), ref, size)
    for out in (model(q, k, v, lk.THIRD, sees, near_only=True), model(q, k, v, lk.THIRD, sees, blind_join=True),
                model(q, k, v, lk.THIRD, sees, taken(m, slice(0, 64), 0)),
                model(q, k, v, lk.THIRD, sees, taken(m, slice(64, 128), 2)), torch.zeros_like(q)):
        with pytest.raises(AssertionError):
            lk.check_thirds(out, ref, size)


def test_a_page_that_is_missing():
    """Its keys outscore all others and have large values: any weight on them shows."""
    m, H, D = 9000, 4, 64
    q, k, v = lk.normal(1, 1, H, D), lk.normal(2, m, H, D), lk.normal(3, m, H, D)
    dead = torch.zeros(m, dtype=torch.bool)
    dead[130 * 64:131 * 64] = True
    q[..., 0], k[..., 0] = 8.0, 0.0
    k[dead, :, 0], v[dead] = 16.0, 100.0
    sees = lk.visible(1, m, True, dead)
    ref, _ = lk.exact(q, k, v, D ** -0.5, sees)
    lk.check_rms(model(q, k, v, D ** -0.5, sees), ref)
    for wrong in (lk.visible(1, m, True), sees | (torch.arange(m) == 130 * 64), sees & (torch.arange(m) // 64 != 129)):
        with pytest.raises(AssertionError):
            lk.check_rms(model(q, k, v, D ** -0.5, wrong), ref)
    zeroed = v.clone()
    zeroed[dead] = 0                                     # the mask left out, the values taken as zeros
    with pytest.raises(AssertionError):
        lk.check_rms(model(q, k, zeroed, D ** -0.5, lk.visible(1, m, True)), ref)

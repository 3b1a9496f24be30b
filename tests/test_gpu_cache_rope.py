"""The norm and rotary turn into the cache against 64-bit plain forms.

A turned value is x c - y s of two normed values x, y with |x| + |y| =: w.  Each carries: its sum of
squares (D terms, fp32: (D / 2) 2^-23 relative after the root), root, division and two products
(6 roundings, 2^-24 each); the turn adds three roundings.  (D / 2 + 16) 2^-23 w covers them; then
one rounding of the result to bf16: 2^-8 of it.  Without a norm the same bound holds.
"""
import numpy as np
import pytest
import torch

import bit_diffusion_transformer_amd as bdt
from tests.helpers import DEV

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
EPS = 1e-6


def ints(x):
    return torch.tensor(np.asarray(x, np.int32), device=DEV)


def inputs(T, H, G, D, R, page, P, norm, seed, spare=2):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def r(*s):
        return torch.randn(s, generator=g, device=DEV)
    rng = np.random.default_rng(seed)
    pages = -(-T // page) + spare
    angle = 60.0 * r(P, R // 2)
    return dict(
        qkv=(r(T, (H + 2 * G) * D) * (0.2 + 2 * torch.rand((H + 2 * G) * D, generator=g, device=DEV))).to(BF),
        gamma_q=(1 + 0.3 * r(D)).to(BF) if norm else None, gamma_k=(1 + 0.3 * r(D)).to(BF) if norm else None,
        cos_t=angle.cos(), sin_t=angle.sin(), positions=ints(rng.integers(0, P, T)),
        slots=ints(rng.permutation(pages * page)[:T]),
        k_cache=torch.full((pages, G, page, D), -777.0, dtype=BF, device=DEV),
        v_cache=torch.full((pages, G, page, D), -555.0, dtype=BF, device=DEV))


def turned_64(x, gamma, cos, sin, R, half):
    """x [T, heads, D] -> (turned, w) fp64; cos, sin [T, R / 2]."""
    x = x.double()
    if gamma is not None:
        x = x / (x.square().mean(-1, keepdim=True) + EPS).sqrt() * gamma.double()
    c, s = cos.double()[:, None], sin.double()[:, None]
    y, w = x.clone(), x.abs()
    first, second = (slice(0, R // 2), slice(R // 2, R)) if half else (slice(0, R, 2), slice(1, R, 2))
    a, b = x[..., first], x[..., second]
    y[..., first], y[..., second] = a * c - b * s, a * s + b * c
    w[..., first] = w[..., second] = a.abs() + b.abs()
    return y, w


def call(i, H, G, half, out=None):
    return bdt.qkv_norm_rope_cache(i["qkv"], H, G, i["gamma_q"], i["gamma_k"], EPS, i["cos_t"], i["sin_t"],
                                   i["positions"], i["slots"], i["k_cache"], i["v_cache"], half=half, out=out)


def check(got, want, w, D, what):
    err = (got.double() - want).abs()
    tol = 2.0 ** -8 * want.abs() + (D / 2 + 16) * 2.0 ** -23 * w
    assert bool((err <= tol + 1e-30).all()), "%s: worst %.3g of the bound" % (what, float((err / (tol + 1e-30)).max()))


CASES = [
    # T, H, G, D, R, page, P
    (1, 1, 1, 64, 16, 16, 1), (1, 32, 8, 128, 128, 64, 900), (7, 3, 1, 128, 48, 16, 50),
    (64, 32, 8, 128, 64, 16, 9000), (333, 5, 5, 64, 64, 32, 333), (129, 12, 4, 128, 112, 256, 10),
    (1000, 8, 2, 64, 48, 128, 2000), (31, 7, 7, 64, 32, 64, 64), (2, 64, 1, 128, 96, 16, 3),
]


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("T,H,G,D,R,page,P", CASES)
def test_norm_and_turn_into_the_cache(T, H, G, D, R, page, P, norm, half):
    i = inputs(T, H, G, D, R, page, P, norm, T + D)
    q = call(i, H, G, half)
    pos, slot = i["positions"].long(), i["slots"].long()
    c, s = i["cos_t"][pos], i["sin_t"][pos]
    x = i["qkv"].view(T, H + 2 * G, D)
    want, w = turned_64(x[:, :H], i["gamma_q"], c, s, R, half)
    check(q, want, w, D, "q")
    want, w = turned_64(x[:, H:H + G], i["gamma_k"], c, s, R, half)
    check(i["k_cache"][slot // page, :, slot % page], want, w, D, "k")
    assert torch.equal(i["v_cache"][slot // page, :, slot % page], x[:, H + G:])
    for cache, left in ((i["k_cache"], -777), (i["v_cache"], -555)):       # other rows stay
        flat = cache.transpose(1, 2).reshape(-1, G * D).clone()
        flat[slot] = left
        assert bool((flat == left).all())


def test_neighbours_agree_with_the_dense_form():
    """The whole head, pairs of neighbours, as many key heads: the values of qkv_norm_rope."""
    T, H, D = 70, 6, 128
    i = inputs(T, H, H, D, D, 16, T, True, 1)
    i["positions"] = ints(range(T))
    q = call(i, H, H, False)
    Q, K, V = bdt.qkv_norm_rope(i["qkv"], H, D, T, i["gamma_q"], i["gamma_k"], EPS, i["cos_t"], i["sin_t"])
    slot = i["slots"].long()
    assert torch.equal(q, Q[0].transpose(0, 1))
    assert torch.equal(i["k_cache"][slot // 16, :, slot % 16], K[0].transpose(0, 1))
    assert torch.equal(i["v_cache"][slot // 16, :, slot % 16], V[0].transpose(0, 1))


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("D", [64, 128])
def test_slots_and_positions_outside(D, half):
    T, H, G, page = 40, 4, 2, 16
    i = inputs(T, H, G, D, 32, page, 50, True, 5)
    pages = i["k_cache"].shape[0]
    ref = {n: (x.clone() if isinstance(x, torch.Tensor) else x) for n, x in i.items()}
    want = call(ref, H, G, half)
    slots, pos = i["slots"].cpu(), i["positions"].cpu()
    for t, x in ((0, -1), (3, pages * page), (17, 2 ** 31 - 1), (39, -2 ** 31)):
        slots[t] = x
    for t, x in ((5, -1), (17, 50), (20, 2 ** 31 - 1), (38, -2 ** 31)):
        pos[t] = x
    i["slots"], i["positions"] = slots.to(DEV), pos.to(DEV)
    out = torch.full_like(want, -111.0)
    call(i, H, G, half, out=out)
    keep = torch.ones(T, dtype=torch.bool)
    keep[[5, 17, 20, 38]] = False
    assert torch.equal(out[keep.to(DEV)], want[keep.to(DEV)])
    assert bool((out[~keep.to(DEV)] == -111).all())
    old = ref["slots"].long()
    for cache, full, left in ((i["k_cache"], ref["k_cache"], -777), (i["v_cache"], ref["v_cache"], -555)):
        expect = full.clone()
        for t in (0, 3, 39, 5, 17, 20, 38):
            expect[old[t] // page, :, old[t] % page] = left
        assert torch.equal(cache, expect)


def test_offsets_past_32_bits():
    G, page, D, pages = 8, 256, 128, 8300
    i = inputs(3, 8, G, D, 128, 256, 9, True, 1)
    small = {n: (x.clone() if isinstance(x, torch.Tensor) else x) for n, x in i.items()}
    small["slots"] = ints([5, 6, 7])
    q = call(small, 8, G, True)
    i["k_cache"] = torch.zeros(pages, G, page, D, dtype=BF, device=DEV)
    i["v_cache"] = torch.zeros_like(i["k_cache"])
    assert i["k_cache"].numel() > 1 << 31
    at = (pages - 2) * page + 5
    i["slots"] = ints([at, at + 1, at + 2])
    assert torch.equal(call(i, 8, G, True), q)
    for n in ("k_cache", "v_cache"):
        assert torch.equal(i[n][pages - 2, :, 5:8], small[n][0, :, 5:8])


def test_values_that_are_not_finite_and_replays():
    T, H, G, D = 9, 4, 2, 128
    i = inputs(T, H, G, D, 128, 16, 20, True, 8)
    clean = call(i, H, G, True)
    kc = i["k_cache"].clone()
    i["qkv"][4, 2 * D + 9] = float("nan")                 # a query head of token 4
    i["qkv"][4, (H + 1) * D + 9] = float("inf")           # a key head
    out = call(i, H, G, True)
    assert bool(out[4, 2].isnan().all())
    out[4, 2] = clean[4, 2]
    assert torch.equal(out, clean)
    s = int(i["slots"][4])
    row = i["k_cache"][s // 16, :, s % 16]
    assert not bool(torch.isfinite(row[1]).all())
    assert torch.equal(row[0], kc[s // 16, :, s % 16][0])
    i["qkv"][4] = 0.0                                     # no length: eps alone
    assert bool((call(i, H, G, True)[4] == 0).all())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q = call(i, H, G, True)
    for it in range(4):
        i["qkv"].copy_(torch.randn(i["qkv"].shape, device=DEV).to(BF))
        i["slots"].copy_(ints(np.random.default_rng(it).permutation(3 * 16)[:T]))
        i["k_cache"].zero_()
        graph.replay()
        torch.cuda.synchronize()
        replayed = q.clone(), i["k_cache"].clone(), i["v_cache"].clone()
        i["k_cache"].zero_()
        eager = call(i, H, G, True)
        assert all(torch.equal(x, y) for x, y in zip(replayed, (eager, i["k_cache"], i["v_cache"])))


def test_empty():
    i = inputs(1, 2, 1, 64, 16, 16, 4, True, 1)
    for n in ("qkv", "positions", "slots"):
        i[n] = i[n][:0].contiguous()
    assert call(i, 2, 1, False).shape == (0, 2, 64)
    i = inputs(5, 2, 1, 64, 16, 16, 4, True, 1)
    i["k_cache"], i["v_cache"] = i["k_cache"][:0].contiguous(), i["v_cache"][:0].contiguous()
    assert call(i, 2, 1, False).shape == (5, 2, 64)       # nothing to cache

"""Block attention where the answer is known beforehand: scores of any magnitude, query rows
that are not finite, values that are not finite.

Large scores.  Every score is exact in fp32 (one power of two times a small whole number, or
sums of whole numbers below 2^24), so softmax(scale s) has no error to inherit from s, however
large.  A key that leads by more than 150 / scale takes all of its row: its weight is 1, the
others' underflow to zero, and the output is its v to the bit.

Where several keys share a row (w = sum p |v|): numerator and denominator use weights rounded
to bf16, 2^-8 of w and of |o|, the result is rounded to bf16, 2^-8 of |o|; fp32 sums over n
keys, 2 n 2^-23 of w; 2^-12 of w for the exponent (the difference s - m is exact; its product
with scale log2 e is off by at most 3 2^-24 of a magnitude below 150), the exponential, the
rescaling and the reciprocal.
"""
import pytest
import torch

import bit_diffusion_transformer_amd as bdt
from bit_diffusion_transformer_amd import _attention
from tests.helpers import DEV
from tests.test_gpu_sparse_attention import attention_64, check, inputs

pytestmark = pytest.mark.gpu
KB = 64
# Sq, keep, kv_len, split over the keys
FORMS = [(1, 32, 2000, True), (400, 32, 2000, True), (1, 1, 61, False), (400, 1, 64, False),
         (1, 32, 70, True)]


def _every(B, H, Sq, keep):
    return torch.arange(keep, dtype=torch.int32, device=DEV).expand(B, H, -(-Sq // 128), keep).contiguous()


def _attend(q, k, v, keep, n, scale, split):
    s = _attention._shape(q, k, None, keep, 0)
    assert (bdt.svdq_block_attention_workspace_bytes(s) > 0) == split
    kv_len = torch.full((q.shape[0],), n, dtype=torch.int32, device=DEV)
    return bdt.block_attention(q, k, v, _every(q.shape[0], q.shape[1], q.shape[2], keep), scale, kv_len)


def _values(G, Sk, D, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(1, G, Sk, D, generator=g, device=DEV).to(torch.bfloat16)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Sq,keep,n,split", FORMS)
@pytest.mark.parametrize("power", [10, 20, 24, 28, 33, 60, 120])
def test_one_leading_key_takes_its_row(D, Sq, keep, n, split, power):
    H, Sk, scale = 2, keep * KB, 0.3
    q = torch.zeros(1, H, Sq, D, dtype=torch.bfloat16, device=DEV)
    q[..., 5] = torch.where(torch.arange(Sq) % 3 == 1, 2.0 ** power, 1.5 * 2.0 ** power).to(DEV)
    k = torch.full((1, H, Sk, D), 0.25, dtype=torch.bfloat16, device=DEV)
    lead = [n // 3, n - 1]
    for h, at in enumerate(lead):
        k[0, h, at, 5] = 1.25
    v = _values(H, Sk, D, power)
    out = _attend(q, k, v, keep, n, scale, split)
    for h, at in enumerate(lead):
        assert torch.equal(out[0, :, h], v[0, h, at].expand(Sq, D)), "head %d" % h


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Sq,keep,n,split", FORMS)
@pytest.mark.parametrize("power", [10, 33, 110])
def test_the_last_of_rising_maxima_and_two_equal_ones(D, Sq, keep, n, split, power):
    """Head 0: the maximum moves with every block.  Head 1: two keys lead by the same score, in
    the first and the last block (the same one where there is only one)."""
    H, Sk = 2, keep * KB
    q = torch.zeros(1, H, Sq, D, dtype=torch.bfloat16, device=DEV)
    q[..., 0] = 2.0 ** power
    k = torch.full((1, H, Sk, D), -1.0, dtype=torch.bfloat16, device=DEV)
    blocks = -(-n // KB)
    for j in range(blocks):
        k[0, 0, min(j * KB + 7 * j % KB, n - 1), 0] = float(j + 1)
    last = min((blocks - 1) * KB + 7 * (blocks - 1) % KB, n - 1)
    a, b = 3, n - 1
    k[0, 1, a, 0] = k[0, 1, b, 0] = 2.0
    v = _values(H, Sk, D, power + 1)
    out = _attend(q, k, v, keep, n, 0.7, split)
    assert torch.equal(out[0, :, 0], v[0, 0, last].expand(Sq, D))
    x, y = v[0, 1, a].double(), v[0, 1, b].double()
    tol = 2.0 ** -8 * ((x + y) / 2).abs() + 2.0 ** -23 * (x.abs() + y.abs())
    assert bool(((out[0, :, 1].double() - (x + y) / 2).abs() <= tol).all())


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Sq,keep,n,split", FORMS)
@pytest.mark.parametrize("offset", [0, 2 ** 10, -2 ** 13, 2 ** 20, -2 ** 22])
def test_a_common_offset_of_the_scores_changes_nothing(D, Sq, keep, n, split, offset):
    """Scores offset + (-40 .. 40), whole numbers below 2^24: softmax does not see the offset."""
    H, Sk = 2, keep * KB
    g = torch.Generator(device=DEV).manual_seed(D + Sq)
    part = torch.randint(-40, 41, (1, H, Sk), generator=g, device=DEV)
    q = torch.zeros(1, H, Sq, D, dtype=torch.bfloat16, device=DEV)
    k = torch.zeros(1, H, Sk, D, dtype=torch.bfloat16, device=DEV)
    q[..., 0], k[..., 0] = float(offset), 1.0
    q[..., 17], k[..., 17] = 1.0, part.to(torch.bfloat16)
    v = _values(H, Sk, D, 3)
    out = _attend(q, k, v, keep, n, 1.0, split)
    p = torch.softmax(part[:, :, :n].double(), dim=-1)
    vd = v[:, :, :n].double()
    o, w = [(p[..., None] * x).sum(2)[:, None] for x in (vd, vd.abs())]      # [1, 1, H, D]
    tol = 2.0 ** -8 * (2 * o.abs() + w) + w * (2 * n * 2.0 ** -23 + 2.0 ** -12)
    assert bool((tol < w / 16).all())
    err = (out.double() - o).abs()
    assert bool((err <= tol).all()), "worst %.3g of the bound" % float((err / tol).max())


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Sq,keep,n,split", FORMS)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_query_row_that_is_not_finite_gives_nan(D, Sq, keep, n, split, bad):
    """And only that row; without any key it gives zeros like every other."""
    H, Sk = 2, keep * KB
    q, k, v = inputs(1, H, H, D, Sq, Sk, 11)
    row = Sq // 2
    clean = q.clone()
    q[0, 1, row] = bad
    out = _attend(q, k, v, keep, n, D ** -0.5, split)
    assert bool(out[0, row, 1].isnan().all())
    out[0, row, 1] = 0
    ref, tol = attention_64(clean, k, v, _every(1, H, Sq, keep).cpu(), D ** -0.5, [n])
    ref[0, row, 1], tol[0, row, 1] = 0, 0
    check(out, ref, tol, "the other rows")
    assert bool((_attend(q, k, v, keep, 0, D ** -0.5, split) == 0).all())


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Sq,keep,n,split", FORMS)
def test_an_infinite_value_of_the_last_key(D, Sq, keep, n, split):
    """v of the last key infinite in some columns: so is the output there, whatever lies behind
    the sequence's length; a NaN gives NaN; the other columns do not change."""
    H, Sk = 2, keep * KB
    q, k, v = inputs(1, H, H, D, Sq, Sk, 12)
    q[...] = 0                                                    # every key counts
    clean = _attend(q, k, v, keep, n, 1.0, split)
    v[:, :, n:] = float("nan")
    v[:, :, n - 1, 3], v[:, :, n - 1, 40], v[:, :, n - 1, 63] = float("inf"), -float("inf"), float("nan")
    out = _attend(q, k, v, keep, n, 1.0, split)
    assert bool((out[..., 3] == float("inf")).all()) and bool((out[..., 40] == -float("inf")).all())
    assert bool(out[..., 63].isnan().all())
    rest = torch.ones(D, dtype=torch.bool, device=DEV)
    rest[[3, 40, 63]] = False
    assert torch.equal(out[..., rest], clean[..., rest])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Sq,keep,n,split", FORMS)
def test_a_key_that_is_nan(D, Sq, keep, n, split):
    """NaN in every row of its head (all take it), in no row of the other; behind the length it
    takes no part."""
    H, Sk = 2, keep * KB
    q, k, v = inputs(1, H, H, D, Sq, Sk, 13)
    clean = _attend(q, k, v, keep, n, D ** -0.5, split)
    k[:, :, n:] = float("nan")
    assert torch.equal(_attend(q, k, v, keep, n, D ** -0.5, split), clean)
    k[0, 1, n // 2, 9] = float("nan")
    out = _attend(q, k, v, keep, n, D ** -0.5, split)
    assert bool(out[:, :, 1].isnan().all()) and torch.equal(out[:, :, 0], clean[:, :, 0])

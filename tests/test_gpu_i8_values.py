"""The 8-bit linear on values that are not finite: they show in the outputs of their own row,
and nowhere else."""
import pytest
import torch

import bit_diffusion_transformer_amd as bdt
from tests.helpers import DEV

pytestmark = pytest.mark.gpu
BAD = [float("nan"), float("inf"), -float("inf")]


def _weights(N, K, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return bdt.i8_pack_weights(torch.randn(N, K, generator=g, device=DEV) * K ** -0.5)


# the form for a few tokens (one, two, four, eight pieces a thread; 8, 16, 32 channels a
# workgroup), a row in registers (each count of pieces), one row or several a workgroup, long rows
@pytest.mark.parametrize("M,N,K", [(1, 72, 64), (2, 2048, 2048), (3, 4096, 1088), (1, 16400, 4096),
                                   (2, 136, 8192), (9, 64, 1024), (40, 1024, 4096), (5, 64, 8192),
                                   (6, 64, 12288), (3, 64, 16384), (3, 64, 16448), (2100, 128, 320),
                                   (4099, 64, 128)])
@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("smooth,act", [(False, 1), (True, 0)])
def test_a_token_that_is_not_finite(M, N, K, bad, smooth, act):
    g = torch.Generator(device=DEV).manual_seed(M + K)
    X = torch.randn(M, K, generator=g, device=DEV).to(torch.bfloat16)
    lam = 0.5 + torch.rand(K, generator=g, device=DEV) if smooth else None
    qw, sw = _weights(N, K, 3)
    bias = torch.randn(N, generator=g, device=DEV).to(torch.bfloat16)
    clean, (qa0, sa0) = bdt.i8_linear(X, lam, qw, sw, bias, act), bdt.i8_quantize_act(X, lam)
    for row, at in ((0, 0), (M // 2, K // 2 + 13), (M - 1, K - 1)):
        Xb = X.clone()
        Xb[row, at] = bad
        Y, (qa, sa) = bdt.i8_linear(Xb, lam, qw, sw, bias, act), bdt.i8_quantize_act(Xb, lam)
        assert bool(Y[row].isnan().all()), "row %d" % row
        assert not bool(sa[row].isfinite()) and not bool(qa[row].any())
        keep = torch.arange(M, device=DEV) != row
        assert torch.equal(Y[keep], clean[keep])
        assert torch.equal(qa[keep], qa0[keep]) and torch.equal(sa[keep], sa0[keep])


@pytest.mark.parametrize("N,K", [(40, 320), (16, 16448), (2056, 128)])
@pytest.mark.parametrize("bad", BAD)
def test_a_channel_that_is_not_finite(N, K, bad):
    g = torch.Generator(device=DEV).manual_seed(N)
    W = torch.randn(N, K, generator=g, device=DEV)
    X = torch.randn(20, K, generator=g, device=DEV).to(torch.bfloat16)
    clean = bdt.i8_linear(X, None, *bdt.i8_pack_weights(W))
    W[7, K - 2] = bad
    Y = bdt.i8_linear(X, None, *bdt.i8_pack_weights(W))
    keep = torch.arange(N, device=DEV) != 7
    assert bool(Y[:, 7].isnan().all()) and torch.equal(Y[:, keep], clean[:, keep])


def test_more_than_2_to_the_23_rows():
    """Each row for itself: slices from both ends and the middle, quantized alone, agree."""
    M, K = (1 << 23) + 5, 64
    g = torch.Generator(device=DEV).manual_seed(1)
    X = torch.randn(M, K, generator=g, device=DEV, dtype=torch.float32).to(torch.bfloat16)
    qa, sa = bdt.i8_quantize_act(X)
    for at in (0, (1 << 22) - 100, (1 << 23) - 100, M - 300):
        q, s = bdt.i8_quantize_act(X[at:at + 300])
        assert torch.equal(qa[at:at + 300], q) and torch.equal(sa[at:at + 300], s)
    assert bool((sa > 0).all())


@pytest.mark.parametrize("M,N,K", [(4128, 960, 320), (4128, 952, 64), (9300, 440, 192)])
@pytest.mark.parametrize("act", [0, 1])
def test_gemm_where_two_narrow_tiles_fit_a_compute_unit(M, N, K, act):
    """Tiles of 128 x 128 just miss one for each compute unit, those of 128 x 64 fit twice."""
    from tests.test_gpu_i8 import _codes, check_y, y_64
    g = torch.Generator(device=DEV).manual_seed(M + N)
    qa, qw = _codes(M, K, 1), _codes(N, K, 2)
    sa, sw = torch.rand(M, generator=g, device=DEV) * 0.02, torch.rand(N, generator=g, device=DEV) * 0.02
    bias = torch.randn(N, generator=g, device=DEV).to(torch.bfloat16)
    ref, mag = y_64(qa, sa, qw, sw, bias, act)
    check_y(bdt.i8_gemm(qa, sa, qw, sw, bias, act), ref, mag, act, "M%d N%d K%d" % (M, N, K))

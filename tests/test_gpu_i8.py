"""The 8-bit linear against 64-bit plain forms.

Codes and scales are bit-exact (the definition's single fp32 steps, done in numpy fp32).
The product's integer sums are exact, so Y differs from the 64-bit value of
act(S sa sw + bias) by: S to fp32, sa sw, their product and the bias sum, each at most
2^-24 relative of its result (the first three move S sa sw by 3 2^-24); GELU, whose slope is
below 1.13, within 4e-7 |y| of the exact form; and one rounding to bf16, 2^-8 relative.
"""
import numpy as np
import pytest
import torch

import bit_diffusion_transformer_amd as bdt
from synth import bf16_bits_to_f32
from tests.helpers import DEV, bf16_f64, bf16_host

pytestmark = pytest.mark.gpu


def quant_np(x: np.ndarray):
    """Codes int8 and scales fp32 of fp32 rows, each step a single fp32 operation."""
    x = x.astype(np.float32)
    with np.errstate(divide="ignore", over="ignore", invalid="ignore"):
        s = (np.abs(x).max(axis=1) / np.float32(127)).astype(np.float32)
        inv = (np.float32(1) / s).astype(np.float32)
        inv[~np.isfinite(inv)] = 0
        q = np.rint((x * inv[:, None]).astype(np.float32))
    return q.astype(np.int8), s


def smooth_np(x, lam):
    if lam is None:
        return x.astype(np.float32)
    return (x.astype(np.float32) * (np.float32(1) / lam).astype(np.float32)).astype(np.float32)


def _acts(M, K, seed, loud=True):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((M, K)).astype(np.float32)
    if loud:
        x[:, rng.random(K) < 0.02] *= 30
    X = torch.from_numpy(x).to(torch.bfloat16)
    lam = rng.uniform(0.2, 4.0, K).astype(np.float32)
    return X, lam


@pytest.mark.parametrize("M,K", [(1, 64), (3, 128), (5, 2048), (7, 2112), (2, 4096), (9, 4160),
                                 (2, 8192), (3, 16384), (2, 16448), (1, 131072), (2049, 192),
                                 (4099, 320)])
@pytest.mark.parametrize("smooth", [False, True])
def test_quantize_act_bit_exact(M, K, smooth):
    X, lam = _acts(M, K, M + K)
    X[M // 2] = 0                                               # a zero row: codes and scale 0
    if M > 2:
        X[0] = torch.full((K,), 1e-40).to(torch.bfloat16)       # 1/s overflows: codes 0
    lam = lam if smooth else None
    qa, sa = bdt.i8_quantize_act(X.to(DEV), None if lam is None else torch.from_numpy(lam).to(DEV))
    q, s = quant_np(smooth_np(bf16_bits_to_f32(bf16_host(X)), lam))
    assert np.array_equal(sa.cpu().numpy().view(np.uint32), s.view(np.uint32))
    assert np.array_equal(qa.cpu().numpy(), q)


def test_quantize_ties_round_to_even():
    K = 64
    x = np.zeros((1, K), np.float32)
    x[0, :6] = [127, 0.5, 1.5, 2.5, -0.5, -3.5]                 # scale 1: exact halves
    qa, sa = bdt.i8_quantize_act(torch.from_numpy(x).to(torch.bfloat16).to(DEV))
    assert qa.cpu().numpy()[0, :6].tolist() == [127, 0, 2, 2, 0, -4] and float(sa[0]) == 1.0


@pytest.mark.parametrize("N,K", [(8, 64), (40, 320), (16, 16448), (4104, 128)])
def test_pack_weights_bit_exact(N, K):
    W = np.random.default_rng(N + K).standard_normal((N, K)).astype(np.float32)
    W[1] = 0
    qw, sw = bdt.i8_pack_weights(torch.from_numpy(W).to(DEV))
    q, s = quant_np(W)
    assert np.array_equal(qw.cpu().numpy(), q)
    assert np.array_equal(sw.cpu().numpy().view(np.uint32), s.view(np.uint32))


def y_64(qa, sa, qw, sw, bias, act):
    """(value, |S sa sw| + |bias|) in 64 bits."""
    t = (qa.double() @ qw.double().t()) * sa.double()[:, None] * sw.double()[None, :]
    y = t if bias is None else t + bias.double()[None, :]
    if act:
        y = y * torch.special.erfc(-y / 2 ** 0.5) / 2
    return y, t.abs() + (0.0 if bias is None else bias.double().abs()[None, :])


def check_y(Y, ref, mag, act, what):
    tol = 2.0 ** -8 * ref.abs() + 1.13 * (4 * 2.0 ** -24) * mag
    if act:
        tol = tol + 4e-7 * mag
    tol = tol + 2.0 ** -24 * mag + 1e-37
    err = (Y.double() - ref).abs()
    assert bool((err <= tol).all()), "%s: worst %.3g of the bound" % (what, float((err / tol).max()))


def _codes(M, K, seed, full=False):
    g = torch.Generator(device=DEV).manual_seed(seed)
    if full:
        return torch.full((M, K), 127, dtype=torch.int8, device=DEV)
    return torch.randint(-127, 128, (M, K), generator=g, device=DEV, dtype=torch.int16).to(torch.int8)


# one row to several tiles of every size, odd row counts, edges in N, K of one half stage up,
# odd and even counts of 64, and shapes that choose each tile size
SHAPES = [(1, 8, 64), (1, 4096, 128), (1, 264, 4096), (2, 64, 192), (15, 72, 320), (16, 128, 64),
          (17, 200, 448), (33, 328, 1024), (64, 64, 576), (65, 1032, 192), (127, 520, 704),
          (128, 2048, 256), (129, 136, 2048), (255, 1000, 64), (257, 4104, 128), (300, 300 * 8, 320),
          (1000, 1000, 1088), (2048, 2048, 512), (2049, 2056, 192), (4000, 4104, 320),
          (4097, 4352, 128), (5, 24, 131072), (64, 8192, 320), (61, 8184, 64), (120, 8200, 1216),
          (630, 4096, 192), (601, 4104, 704), (1000, 4096, 448), (2040, 4096, 320), (2990, 4096, 192),
          (4096, 4096, 256), (4601, 4096, 512), (4608, 4088, 64), (7, 1000, 448), (3, 40, 576)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("act", [0, 1])
def test_gemm(M, N, K, act):
    g = torch.Generator(device=DEV).manual_seed(M * 3 + N)
    qa, qw = _codes(M, K, 1 + M), _codes(N, K, 2 + N)
    sa = torch.rand(M, generator=g, device=DEV) * 0.02
    sw = torch.rand(N, generator=g, device=DEV) * 0.02
    bias = torch.randn(N, generator=g, device=DEV).to(torch.bfloat16) if (M + act) % 2 else None
    Y = bdt.i8_gemm(qa, sa, qw, sw, bias, act)
    ref, mag = y_64(qa, sa, qw, sw, bias, act)
    check_y(Y, ref, mag, act, "M%d N%d K%d" % (M, N, K))
    assert torch.equal(Y, bdt.i8_gemm(qa, sa, qw, sw, bias, act))     # deterministic


@pytest.mark.parametrize("M", [4, 300, 4096])
def test_gelu_epilogue_accuracy(M):
    """One product of 127 127 per output, scaled to a grid of pre-activations over -12 .. 12, the
    tails and zero, on every tile size: half a bf16 step and 4e-7 |x| of the exact erf form
    (the pre-activation itself is off by at most 2 2^-24 of it, and GELU's slope is below 1.13)."""
    K, N = 64, 4096
    x = torch.cat([torch.linspace(-12, 12, N - 40, dtype=torch.float64, device=DEV),
                   torch.logspace(-30, 30, 20, dtype=torch.float64, device=DEV),
                   -torch.logspace(-30, 30, 20, dtype=torch.float64, device=DEV)])
    qa = torch.zeros(M, K, dtype=torch.int8, device=DEV)
    qw = torch.zeros(N, K, dtype=torch.int8, device=DEV)
    qa[:, 0], qw[:, 0] = 127, 127
    sw = (x / 16129).float()
    Y = bdt.i8_gemm(qa, torch.ones(M, device=DEV), qw, sw, None, 1).double()
    pre = sw.double() * 16129
    ref = pre * torch.special.erfc(-pre / 2 ** 0.5) / 2
    tol = 2.0 ** -8 * ref.abs() + (4e-7 + 1.13 * 2 * 2.0 ** -24) * pre.abs()
    assert bool(((Y - ref).abs() <= tol).all())


@pytest.mark.parametrize("M", [1, 4, 40, 300, 2100, 4096])
def test_gelu_of_what_is_not_finite(M):
    """NaN stays NaN, +inf stays, -inf goes to the limit 0 (held at |x| = 8, where GELU is below
    8 2^-50); the columns beside them are untouched."""
    K, N = 64, 2048
    qa, qw = _codes(M, K, 3), _codes(N, K, 4)
    sa, sw = torch.full((M,), 0.01, device=DEV), torch.full((N,), 0.01, device=DEV)
    bias = torch.zeros(N, dtype=torch.bfloat16, device=DEV)
    bad = bias.clone()
    bad[5::64], bad[6::64], bad[7::64] = float("nan"), float("inf"), -float("inf")
    X, _ = _acts(M, K, 8)
    for run in (lambda b: bdt.i8_gemm(qa, sa, qw, sw, b, 1), lambda b: bdt.i8_linear(X.to(DEV), None, qw, sw, b, 1)):
        Y, clean = run(bad), run(bias)
        assert bool(Y[:, 5::64].isnan().all()) and bool((Y[:, 6::64] == float("inf")).all())
        assert bool((Y[:, 7::64].abs() <= 8 * 2.0 ** -50).all())
        keep = torch.ones(N, dtype=torch.bool, device=DEV)
        for i in (5, 6, 7):
            keep[i::64] = False
        assert torch.equal(Y[:, keep], clean[:, keep])


@pytest.mark.parametrize("M", [1, 16, 200, 3000])
def test_gemm_largest_sums_are_exact(M):
    """Every code 127 at the longest K: S = 127^2 2^17, below 2^31 by less than 2 %; scales of
    powers of two leave one rounding (S to bf16)."""
    K, N = 1 << 17, 2048
    qa, qw = _codes(M, K, 0, True), _codes(N, K, 0, True)
    qw[::2] = -127
    one = torch.ones(N, device=DEV)
    Y = bdt.i8_gemm(qa, torch.ones(M, device=DEV), qw, one)
    S = torch.tensor(float(127 * 127 * K)).to(torch.bfloat16).item()
    assert bool((Y[:, 1::2] == S).all()) and bool((Y[:, ::2] == -S).all())


@pytest.mark.parametrize("M,N,K", [(1, 512, 256), (37, 264, 1984), (700, 1536, 1024)])
def test_outputs_stay_inside(M, N, K):
    qa, qw = _codes(M, K, 5), _codes(N, K, 6)
    sa, sw = torch.ones(M, device=DEV), torch.ones(N, device=DEV)
    buf = torch.full((M * N + 512,), -777.0, dtype=torch.bfloat16, device=DEV)
    Y = buf[256:256 + M * N].view(M, N)
    need = bdt.svdq_i8_gemm_workspace_bytes(M, N, K)
    ws = torch.full((need + 512,), 0x5A, dtype=torch.uint8, device=DEV)
    bdt.svdq_i8_gemm(qa, sa, qw, sw, None, 0, M, N, K, Y, ws[256:] if need else None, need)
    assert bool((buf[:256] == -777).all()) and bool((buf[256 + M * N:] == -777).all())
    assert bool((ws[:256] == 0x5A).all()) and bool((ws[256 + need:] == 0x5A).all())
    assert torch.equal(Y, bdt.i8_gemm(qa, sa, qw, sw))


@pytest.mark.parametrize("M,N,K,smooth,act", [(1, 1536, 512, True, 0), (13, 136, 4160, False, 1),
                                              (513, 1024, 1024, True, 1), (2500, 2048, 640, True, 0)])
def test_linear_is_its_two_steps(M, N, K, smooth, act):
    X, lam = _acts(M, K, 77)
    X, lam = X.to(DEV), torch.from_numpy(lam).to(DEV) if smooth else None
    g = torch.Generator(device=DEV).manual_seed(3)
    W = torch.randn(N, K, generator=g, device=DEV) * K ** -0.5
    bias = torch.randn(N, generator=g, device=DEV).to(torch.bfloat16)
    qw, sw = bdt.i8_pack_weights(W if lam is None else W * lam)
    qa, sa = bdt.i8_quantize_act(X, lam)
    Y = bdt.i8_linear(X, lam, qw, sw, bias, act)
    assert torch.equal(Y, bdt.i8_gemm(qa, sa, qw, sw, bias, act))
    # and near the unquantized product: 8-bit codes are off by at most half a step of s
    # (of x against |qw sw|, of w against |x| <= (|qa| + 1/2) sa)
    step = sa.double()[:, None] / 2 * (qw.double().abs().sum(1) * sw.double())[None, :] \
        + (sw.double() / 2)[None, :] * (sa.double() * (qa.double().abs().sum(1) + K / 2.0))[:, None]
    full = X.double() @ W.double().t() + bias.double()
    if act:
        full = full * torch.special.erfc(-full / 2 ** 0.5) / 2
    assert bool(((Y.double() - full).abs() <= 1.13 * step * 1.001 + 2.0 ** -8 * full.abs() + 1e-6).all())


@pytest.mark.parametrize("M,N,K", [(1, 8, 64), (1, 40, 192), (2, 264, 2048), (4, 8192, 2048), (4, 8200, 2048),
                                   (1, 8200, 4096), (2, 72, 2112), (3, 72, 2112), (1, 24, 8192),
                                   (1, 1000, 8128), (3, 520, 1984), (2, 16400, 320), (1, 40000, 128),
                                   (1, 4096, 448), (4, 32, 576), (1, 16, 8256), (1, 2040, 2048), (1, 2056, 2048),
                                   (1, 2048, 2112), (4, 4096, 1024), (4, 4104, 1024), (2, 8184, 3968),
                                   (1, 8, 7680), (3, 8, 1728), (1, 4096, 7552), (1, 4096, 16384),
                                   (1, 72, 16448), (2, 136, 8192), (2, 4104, 8192), (2, 520, 4160),
                                   (4, 264, 4096)])
@pytest.mark.parametrize("smooth,act", [(False, 0), (True, 1)])
def test_linear_of_a_few_tokens(M, N, K, smooth, act):
    """One launch or two, by the sizes: the codes, scales and sums are the same, so the outputs
    are; nothing is written outside them."""
    X, lam = _acts(M, K, M + N)
    if M > 1:
        X[1] = 0
    if M > 3:
        X[3] = torch.full((K,), 1e-40).to(torch.bfloat16)
    X, lam = X.to(DEV), torch.from_numpy(lam).to(DEV) if smooth else None
    qw, sw = _codes(N, K, N), torch.rand(N, device=DEV) * 0.02
    bias = torch.randn(N, device=DEV).to(torch.bfloat16) if act else None
    qa, sa = bdt.i8_quantize_act(X, lam)
    want = bdt.i8_gemm(qa, sa, qw, sw, bias, act)
    need = bdt.svdq_i8_linear_workspace_bytes(M, N, K)
    for _ in range(2):
        buf = torch.full((M * N + 512,), -777.0, dtype=torch.bfloat16, device=DEV)
        ws = torch.full((need + 512,), 0x5A, dtype=torch.uint8, device=DEV)
        bdt.svdq_i8_linear(X, lam, qw, sw, bias, act, M, N, K, buf[256:256 + M * N], ws[256:], need)
        assert torch.equal(buf[256:256 + M * N].view(M, N), want)
        assert bool((buf[:256] == -777).all()) and bool((buf[256 + M * N:] == -777).all())
        assert bool((ws[:256] == 0x5A).all()) and bool((ws[256 + need:] == 0x5A).all())


def test_layer_object_is_the_linear():
    g = torch.Generator(device=DEV).manual_seed(6)
    W, lam = torch.randn(72, 320, generator=g, device=DEV), 0.5 + torch.rand(320, generator=g, device=DEV)
    bias = torch.randn(72, generator=g, device=DEV).to(torch.bfloat16)
    X = torch.randn(9, 320, generator=g, device=DEV).to(torch.bfloat16)
    layer = bdt.I8Linear.from_weight(W, lam, bias, bdt.ACT_GELU)
    assert (layer.in_features, layer.out_features) == (320, 72)
    qw, sw = bdt.i8_pack_weights(W * lam)
    assert torch.equal(layer(X), bdt.i8_linear(X, lam, qw, sw, bias, bdt.ACT_GELU))
    plain = bdt.I8Linear.from_weight(W)
    assert torch.equal(plain(X), bdt.i8_linear(X, None, *bdt.i8_pack_weights(W)))


@pytest.mark.parametrize("M", [1, 100, 1100])
def test_linear_in_a_graph_and_on_two_streams(M):
    K, N = 1024, 1536
    X, lam = _acts(M, K, 5)
    X, lam = X.to(DEV), torch.from_numpy(lam).to(DEV)
    qw, sw = _codes(N, K, 9), torch.rand(N, device=DEV) * 0.01
    X2 = X.flip(0).contiguous() * 0.5
    want = bdt.i8_linear(X, lam, qw, sw), bdt.i8_linear(X2, lam, qw, sw)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (s1, s2):
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        with torch.cuda.stream(s1):
            a = bdt.i8_linear(X, lam, qw, sw)
        with torch.cuda.stream(s2):
            b = bdt.i8_linear(X2, lam, qw, sw)
        torch.cuda.synchronize()
        assert torch.equal(a, want[0]) and torch.equal(b, want[1])
    Xg = X.clone()
    with torch.cuda.stream(s1):
        bdt.i8_linear(Xg, lam, qw, sw)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        Y = bdt.i8_linear(Xg, lam, qw, sw)
    for it in range(4):
        Xg.copy_(X if it % 2 else X2)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(Y, want[0 if it % 2 else 1]), "replay %d" % it


def test_empty():
    qw, sw = _codes(16, 128, 1), torch.ones(16, device=DEV)
    assert bdt.i8_linear(torch.empty(0, 128, dtype=torch.bfloat16, device=DEV), None, qw, sw).shape == (0, 16)
    assert bf16_f64(bf16_host(bdt.i8_gemm(qw[:0], sw[:0], qw, sw))).shape == (0, 16)

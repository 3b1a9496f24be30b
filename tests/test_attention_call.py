"""bdt.attention checks every tensor before it launches anything, and runs its three steps on
the tensors' own device.  (The kernels trust the sizes they are given: a table shorter than
the sequence, or a projection narrower than its heads, would be read past its end.)"""
import contextlib

import pytest
import torch

import bit_diffusion_transformer_amd as bdt

B, S, H, D, K, R, N = 2, 6, 2, 64, 192, 16, 40
HD = H * D


def _layer(n_in, n_out, r=R):
    low = dict(L1=torch.zeros(n_in, r, dtype=torch.bfloat16), L2=torch.zeros(r, n_out, dtype=torch.bfloat16))
    return dict(lam=torch.ones(n_in), qw=torch.zeros(bdt.pair_rows(n_out), n_in, dtype=torch.uint8),
                sw=torch.zeros(bdt.scale_shape(n_out, n_in)), bias=torch.zeros(n_out, dtype=torch.bfloat16),
                **(low if r else dict(L1=None, L2=None)))


def _args(**kw):
    bf = torch.bfloat16
    a = dict(X=torch.zeros(B * S, K, dtype=bf), qkv=_layer(K, 3 * HD), out=_layer(HD, N), heads=H,
             head_dim=D, seq=S, gamma_q=torch.ones(D, dtype=bf), gamma_k=torch.ones(D, dtype=bf),
             eps=1e-6, cos_t=torch.ones(S, D // 2), sin_t=torch.zeros(S, D // 2), keep=1,
             kv_len=torch.full((B,), S, dtype=torch.int32))
    a.update(kw)
    return a


def _less(layer, **kw):
    return {**layer, **kw}


@pytest.fixture
def nothing_launched(monkeypatch):
    def refuse(*a, **k):
        raise AssertionError("a step ran")
    for step in ("linear_qkv", "sparse_attention", "linear"):
        monkeypatch.setattr(bdt, step, refuse)


Q, O = _layer(K, 3 * HD), _layer(HD, N)


@pytest.mark.parametrize("kw", [
    dict(cos_t=torch.ones(S - 1, D // 2)), dict(sin_t=torch.ones(S, D // 2 - 1)),
    dict(cos_t=torch.ones(S, D)), dict(gamma_q=torch.ones(D // 2, dtype=torch.bfloat16)),
    dict(gamma_k=torch.ones(2 * D, dtype=torch.bfloat16)), dict(heads=H + 1), dict(heads=2 * H),
    dict(head_dim=128), dict(heads=-H, head_dim=-D), dict(seq=S + 1), dict(seq=0), dict(seq=5),
    dict(X=torch.zeros(B * S, K - 64, dtype=torch.bfloat16)), dict(X=torch.zeros(B, S, K, dtype=torch.bfloat16)),
    dict(kv_len=torch.zeros(B + 1, dtype=torch.int32)),
    dict(qkv=_layer(K, 2 * HD)), dict(qkv=_less(Q, lam=torch.ones(K - 1))),
    dict(qkv=_less(Q, bias=torch.zeros(HD, dtype=torch.bfloat16))),
    dict(qkv=_less(Q, L1=torch.zeros(K - 64, R, dtype=torch.bfloat16))),
    dict(qkv=_less(Q, L2=torch.zeros(R // 2, 3 * HD, dtype=torch.bfloat16))),
    dict(qkv=_less(Q, L2=None)), dict(qkv=_less(Q, sw=torch.zeros(2, 3 * HD))),
    dict(out=_layer(HD + 64, N)), dict(out=_less(O, qw=torch.zeros(N, HD // 2, dtype=torch.uint8))),
    dict(out=_less(O, L2=torch.zeros(R, N - 8, dtype=torch.bfloat16))), dict(out=_less(O, lam=torch.ones(K))),
    dict(out=_less(O, bias=torch.zeros(N + 8, dtype=torch.bfloat16))),
])
def test_sizes_that_do_not_fit_are_refused(nothing_launched, kw):
    with pytest.raises((ValueError, TypeError), match="shape|multiple|tensor"):
        bdt.attention(**_args(**kw))


@pytest.mark.parametrize("kw", [
    dict(X=torch.zeros(B * S, K)), dict(cos_t=torch.ones(S, D // 2).double()), dict(gamma_q=torch.ones(D)),
    dict(kv_len=torch.zeros(B, dtype=torch.int64)), dict(qkv=_less(Q, lam=torch.ones(K).half())),
    dict(out=_less(O, sw=torch.zeros(bdt.scale_shape(N, HD)).double())), dict(gamma_k=None),
    dict(out=_less(O, qw=O["qw"].to(torch.int8))), dict(qkv=_less(Q, bias=torch.zeros(3 * HD))),
])
def test_types_that_do_not_fit_are_refused(nothing_launched, kw):
    with pytest.raises((ValueError, TypeError), match="expected"):
        bdt.attention(**_args(**kw))


def test_tensors_that_are_not_on_a_gpu_are_refused(nothing_launched):
    with pytest.raises(ValueError, match="GPU"):
        bdt.attention(**_args())
    with pytest.raises(ValueError, match="GPU"):
        bdt.attention(**_args(qkv=_layer(K, 3 * HD, 0), out=_layer(HD, N, 0), kv_len=None))
    longer = torch.ones(S + 9, D // 2)                 # rows past seq are not read
    with pytest.raises(ValueError, match="GPU"):
        bdt.attention(**_args(cos_t=longer, sin_t=longer, qkv=_less(Q, name="to_qkv")))
    with pytest.raises(ValueError, match="contiguous"):
        bdt.attention(**_args(X=torch.zeros(K, B * S, dtype=torch.bfloat16).t()))


def test_every_step_runs_on_the_tensors_device(monkeypatch):
    ran, current = [], []

    @contextlib.contextmanager
    def on(dev):
        current.append(dev)
        yield
        current.pop()

    def step(name, out):
        def f(*a, **k):
            ran.append((name, list(current)))
            return out
        return f
    bf = torch.bfloat16
    heads = torch.zeros(B, H, S, D, dtype=bf)
    monkeypatch.setattr(bdt, "one_device", lambda **k: "the device")
    monkeypatch.setattr(bdt, "on", on)
    monkeypatch.setattr(bdt, "linear_qkv", step("qkv", (heads,) * 3))
    monkeypatch.setattr(bdt, "sparse_attention", step("attention", torch.zeros(B, S, H, D, dtype=bf)))
    monkeypatch.setattr(bdt, "linear", step("out", torch.zeros(B * S, N, dtype=bf)))
    assert bdt.attention(**_args()).shape == (B * S, N)
    assert ran == [(n, ["the device"]) for n in ("qkv", "attention", "out")]


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["X", "cos_t", "gamma_k", "kv_len", "qkv", "out"])
def test_a_tensor_left_on_the_host_is_refused(nothing_launched, name):
    def up(v):
        if isinstance(v, dict):
            return {n: up(t) for n, t in v.items()}
        return v.cuda() if isinstance(v, torch.Tensor) else v
    args = _args()
    args = {n: v if n == name else up(v) for n, v in args.items()}
    with pytest.raises(ValueError, match="must be on a GPU"):
        bdt.attention(**args)

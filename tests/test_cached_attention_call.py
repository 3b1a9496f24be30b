"""bdt.cached_attention checks every tensor before it launches anything: its first step writes
the caches, so a later refusal would leave them changed."""
import pytest
import torch

import bit_diffusion_transformer_amd as bdt
from tests.test_attention_call import _layer, _less

H, G, D, K, T, B, N = 4, 2, 64, 192, 6, 3, 40
HD = H * D
BF, I32 = torch.bfloat16, torch.int32


def _args(**kw):
    a = dict(X=torch.zeros(T, K, dtype=BF), qkv=_layer(K, (H + 2 * G) * D), out=_layer(HD, N), heads=H, kv_heads=G,
             head_dim=D, gamma_q=torch.ones(D, dtype=BF), gamma_k=None, eps=1e-6, cos_t=torch.ones(9, D // 2),
             sin_t=torch.zeros(9, D // 2), k_cache=torch.zeros(5, G, 16, D, dtype=BF),
             v_cache=torch.zeros(5, G, 16, D, dtype=BF), tables=torch.zeros(B, 4, dtype=I32),
             q_starts=torch.zeros(B + 1, dtype=I32), kv_len=torch.zeros(B, dtype=I32), slots=torch.zeros(T, dtype=I32),
             positions=torch.zeros(T, dtype=I32))
    a.update(kw)
    return a


@pytest.fixture
def nothing_launched(monkeypatch):
    def refuse(*a, **k):
        raise AssertionError("a step ran")
    for step in ("linear", "qkv_norm_rope_cache", "paged_attention"):
        monkeypatch.setattr(bdt, step, refuse)


Q, O = _layer(K, (H + 2 * G) * D), _layer(HD, N)


@pytest.mark.parametrize("kw", [
    dict(heads=H + 1), dict(kv_heads=G + 1), dict(head_dim=128), dict(X=torch.zeros(T, K - 64, dtype=BF)),
    dict(X=torch.zeros(T + 1, K, dtype=BF)), dict(qkv=_layer(K, 3 * HD)), dict(qkv=_less(Q, lam=torch.ones(K - 1))),
    dict(out=_layer(HD + 64, N)), dict(gamma_q=torch.ones(2 * D, dtype=BF)), dict(gamma_k=torch.ones(8, dtype=BF)),
    dict(sin_t=torch.zeros(8, D // 2)), dict(v_cache=torch.zeros(5, G, 32, D, dtype=BF)),
    dict(tables=torch.zeros(B + 1, 4, dtype=I32)), dict(q_starts=torch.zeros(B, dtype=I32)),
    dict(kv_len=torch.zeros(B + 1, dtype=I32)), dict(slots=torch.zeros(T - 1, dtype=I32)),
    dict(positions=torch.zeros(T + 1, dtype=I32)), dict(X=torch.zeros(T, K)), dict(slots=torch.zeros(T)),
    dict(k_cache=torch.zeros(5, G, 16, D)), dict(tables=torch.zeros(B, 4, dtype=torch.int64)), dict(cos_t=None),
])
def test_what_does_not_fit_is_refused(nothing_launched, kw):
    with pytest.raises((ValueError, TypeError), match="shape|expected"):
        bdt.cached_attention(**_args(**kw))


def test_tensors_that_are_not_on_a_gpu_are_refused(nothing_launched):
    with pytest.raises(ValueError, match="GPU"):
        bdt.cached_attention(**_args())


@pytest.mark.parametrize("most", [0, -1])
def test_a_most_below_one_is_refused(nothing_launched, most):
    with pytest.raises(ValueError, match="max_new"):
        bdt.cached_attention(**_args(), max_new=most)


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["X", "cos_t", "gamma_q", "k_cache", "tables", "kv_len", "slots", "qkv", "out"])
def test_a_tensor_left_on_the_host_is_refused(nothing_launched, name):
    def up(v):
        if isinstance(v, dict):
            return {n: up(t) for n, t in v.items()}
        return v.cuda() if isinstance(v, torch.Tensor) else v
    args = {n: v if n == name else up(v) for n, v in _args().items()}
    with pytest.raises(ValueError, match="must be on a GPU"):
        bdt.cached_attention(**args)

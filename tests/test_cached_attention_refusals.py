"""bdt.cached_attention refuses what any of its four steps would refuse before the first of them
runs: the second step writes the caches."""
import pytest
import torch

import bit_diffusion_transformer_amd as bdt
from tests.test_attention_call import _layer, _less
from tests.test_cached_attention_call import B, BF, D, G, H, HD, I32, K, N, T, _args, nothing_launched  # noqa: F401


def off_by(t):
    """t's values at an address that is 2 or 4 bytes past a 16-byte boundary."""
    flat = torch.zeros(t.numel() + 1, dtype=t.dtype, device=t.device)[1:]
    return flat.copy_(t.flatten()).view(t.shape)


def up(v):
    if isinstance(v, dict):
        return {n: up(t) for n, t in v.items()}
    return v.cuda() if isinstance(v, torch.Tensor) else v


def halves(rotary):
    return dict(cos_t=torch.ones(9, rotary // 2), sin_t=torch.zeros(9, rotary // 2))


def caches(page, g=G, d=D):
    return {n: torch.zeros(5, g, page, d, dtype=BF) for n in ("k_cache", "v_cache")}


def heads(h, g, d):
    """A call that fits together with other heads."""
    return dict(heads=h, kv_heads=g, head_dim=d, qkv=_layer(K, (h + 2 * g) * d), out=_layer(h * d, N),
                gamma_q=torch.ones(d, dtype=BF), cos_t=torch.ones(9, 16), sin_t=torch.zeros(9, 16), **caches(16, g, d))


OUT = _layer(HD, N)
REFUSED = [
    # the last step's
    (dict(out=_layer(HD, N, r=8)), "rank"), (dict(out=_layer(HD, N, r=144)), "rank"), (dict(out=_layer(HD, 36)), "N must"),
    (dict(out=_less(OUT, bias=off_by(OUT["bias"]))), "bias"), (dict(out=_less(OUT, lam=off_by(OUT["lam"]))), "lambda"),
    (dict(out=_less(OUT, L2=off_by(OUT["L2"]))), "L2"), (dict(out=_less(OUT, sw=off_by(OUT["sw"]))), "sw"),
    # the attention's
    (dict(tables=torch.zeros(1, (1 << 26) + 1, dtype=I32), q_starts=torch.zeros(2, dtype=I32),
          kv_len=torch.zeros(1, dtype=I32)), "exceed"), (heads(65, 1, 64), "heads / kv_heads"),
    (heads(4, 3, 64), "divide"), (heads(4, 2, 32), "head_dim"), (dict(max_new=1.5), "int"),
    (dict(k_cache=off_by(torch.zeros(5, G, 16, D, dtype=BF))), "cache"),
    # the norm's and the cache's
    (caches(24), "page"), (caches(8), "page"), (halves(24), "rotary"), (halves(2 * D), "rotary"), (dict(eps=-1.0), "eps"),
    (dict(eps=float("nan")), "eps"), (dict(cos_t=torch.ones(0, 16), sin_t=torch.ones(0, 16)), "table_rows"),
    (dict(gamma_q=off_by(torch.ones(D, dtype=BF))), "gamma"), (dict(cos_t=off_by(torch.ones(9, D // 2))), "rotary"),
]


@pytest.mark.parametrize("kw,match", REFUSED, ids=[str(i) for i in range(len(REFUSED))])
def test_what_a_later_step_refuses_is_refused_first(nothing_launched, kw, match):  # noqa: F811
    with pytest.raises((RuntimeError, ValueError, TypeError), match=match):
        bdt.cached_attention(**_args(**kw))


def test_no_tokens_and_no_requests_pass_the_checks(nothing_launched):  # noqa: F811
    """On the CPU they are refused for being there, and for nothing else."""
    none = torch.zeros(0, dtype=I32)
    for kw in (dict(X=torch.zeros(0, K, dtype=BF), slots=none, positions=none), dict(out=_layer(HD, N, r=0)),
               dict(tables=torch.zeros(0, 4, dtype=I32), q_starts=torch.zeros(1, dtype=I32), kv_len=none),
               caches(256), {n: torch.zeros(0, G, 16, D, dtype=BF) for n in ("k_cache", "v_cache")}, halves(16)):
        with pytest.raises(ValueError, match="GPU"):
            bdt.cached_attention(**_args(**kw))


@pytest.mark.gpu
@pytest.mark.parametrize("kw", [dict(out=_layer(HD, N, r=8)), dict(out=_layer(HD, 36)), dict(max_new=1.5), dict(eps=-1.0)])
def test_the_caches_stay_as_they_were(kw):
    args = {n: up(v) for n, v in _args(k_cache=torch.full((5, G, 16, D), 3.0, dtype=BF),
                                       v_cache=torch.full((5, G, 16, D), 4.0, dtype=BF),
                                       slots=torch.arange(T, dtype=I32), **kw).items()}
    with pytest.raises((RuntimeError, TypeError)):
        bdt.cached_attention(**args)
    assert bool((args["k_cache"] == 3).all()) and bool((args["v_cache"] == 4).all())


@pytest.mark.gpu
def test_no_tokens_and_no_requests_run():
    none = torch.zeros(0, dtype=I32)
    for kw, rows in ((dict(X=torch.zeros(0, K, dtype=BF), slots=none, positions=none), 0),
                     (dict(tables=torch.zeros(0, 4, dtype=I32), q_starts=torch.zeros(1, dtype=I32), kv_len=none), T),
                     ({n: torch.zeros(0, G, 16, D, dtype=BF) for n in ("k_cache", "v_cache")}, T),
                     (dict(tables=torch.zeros(B, 0, dtype=I32)), T)):
        args = {n: up(v) for n, v in _args(**kw).items()}
        assert bdt.cached_attention(**args).shape == (rows, N)
        torch.cuda.synchronize()

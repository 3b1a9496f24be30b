"""Rotary tables at the edge of the stated range, |position| <= 2^26 and theta >= 1, against
80-bit references.

The bound, 2^-21 = 8 u with u = 2^-24: the reduced angle rounded to fp32 in half turns, pi u; the
fp32 sine and cosine, 4 u; and the angle itself.  With v = 2^-53: the logarithm of theta, the
quotient and their product are off by 4 v of a product x log(theta) whose frequency is
theta^-x, and x log(theta) theta^-x <= 1 / e: 1.5 v; the exponential, the factor 1 / 2 pi and the
two products, 5 v: together 6.5 v |position|, below 0.85 u at 2^26.
"""
import numpy as np
import pytest
import torch

import bit_diffusion_transformer_amd as bdt
from tests.helpers import DEV

pytestmark = pytest.mark.gpu


def tables_80(pos, dims, thetas):
    L = np.longdouble
    cols = [pos[:, a:a + 1].astype(L) * np.exp(np.log(L(t)) * (L(-2) * np.arange(d // 2).astype(L) / L(d)))
            for a, (d, t) in enumerate(zip(dims, thetas))]
    angle = np.concatenate(cols, axis=1)
    return np.cos(angle), np.sin(angle)


@pytest.mark.parametrize("dims,thetas", [((16, 56, 56), (1e4,) * 3), ((64, 64), (1.0, 1.5)),
                                         ((128,), (1e6,)), ((32, 32, 32, 32), (2.0, 256.0, 1e9, 1e30)),
                                         ((256,), (500000.0,))])
@pytest.mark.parametrize("most", [2.0 ** 21, 2.0 ** 26])
def test_tables_at_the_edge_of_the_range(dims, thetas, most):
    assert np.finfo(np.longdouble).nmant >= 63
    rng = np.random.default_rng(int(most) % 1000 + len(dims))
    pos = rng.uniform(-most, most, (3001, len(dims))).astype(np.float32)
    pos[:500] = most - 4.0 * np.arange(500)[:, None]
    pos[500:1000] = -pos[:500]
    cos, sin = bdt.rope_tables(torch.from_numpy(pos).to(DEV), dims, thetas)
    c, s = tables_80(pos, dims, thetas)
    assert np.abs(cos.cpu().numpy() - c).max() <= 2.0 ** -21
    assert np.abs(sin.cpu().numpy() - s).max() <= 2.0 ** -21

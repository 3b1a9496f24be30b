"""Values up to the range that include/svdq_paged.h states: the sum of |v| over a row's keys below
2^119.  A power of two on v is one on every product, sum and quotient, so the results are the
same bits but for the exponent."""
import pytest
import torch

import bit_diffusion_transformer_amd as bdt
from tests import long_keys as lk
from tests.helpers import DEV
from tests.test_gpu_paged_long import ints, starts

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("page,H,G,D,new,lens", [(None, 8, 2, 128, [500, 3], [500, 3]), (None, 2, 1, 64, [1000], [1000]),
                                                 (64, 32, 8, 128, [1, 1], [900, 100]), (16, 8, 2, 64, [3, 700], [1000, 701]),
                                                 (32, 6, 2, 128, [150], [800])])
def test_large_values(page, H, G, D, new, lens):
    q = torch.cat([lk.normal(b, n, H, D, device=DEV) for b, n in enumerate(new)])
    ks = [lk.normal(10 + b, m, G, D, device=DEV) for b, m in enumerate(lens)]
    vs = [lk.positive(20 + b, m, G, D, device=DEV) for b, m in enumerate(lens)]     # 1 .. 2, 1000 of them: below 2^11

    def call(gain):
        big = [v * gain for v in vs]
        if page is None:
            return bdt.packed_attention(q, torch.cat(ks), torch.cat(big), ints(starts(new)))
        kc, vc, tables = lk.in_pages(ks, big, page, 3)
        return bdt.paged_attention(q, kc, vc, tables.to(DEV), ints(starts(new)), ints(lens), max_new=max(new))
    small, large = call(1.0), call(2.0 ** 108)
    assert bool(torch.isfinite(large.float()).all())
    assert torch.equal(large, (small.double() * 2.0 ** 108).to(torch.bfloat16))

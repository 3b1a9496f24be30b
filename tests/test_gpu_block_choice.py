"""The choice of key blocks for every number of query blocks that a workgroup takes (16, 8 or
4, by the number of key blocks and of workgroups), against the 64-bit lists; up to 4096 key
blocks, whose scores fill 128 KB of LDS."""
import pytest
import torch

import bit_diffusion_transformer_amd as bdt
from tests.helpers import DEV
from tests.test_gpu_sparse_attention import attention_64, check, inputs, lists_64

pytestmark = pytest.mark.gpu

# B, H, G, D, query blocks (the last one not whole), Sk, keep, first, kv_len
CASES = [
    (1, 24, 24, 64, 88, 1300, 4, 0, None),              # 16 query blocks: the last workgroup has 8
    (2, 40, 8, 64, 33, 700, 3, 1, [700, 449]),          # 16, the last workgroup has one
    (1, 12, 12, 128, 180, 4000, 20, 0, [3999]),         # 16, 63 key blocks
    (1, 10, 2, 128, 209, 32700, 64, 2, None),           # 16, 511 key blocks: 64 KB
    (1, 4, 4, 64, 17, 32768, 70, 0, None),              # 8: a compute unit for each workgroup
    (2, 2, 1, 128, 10, 40000, 10, 1, [40000, 33333]),   # 8: 625 key blocks
    (1, 3, 3, 64, 9, 65536, 5, 0, None),                # 8: 1024, 64 KB
    (1, 2, 2, 64, 6, 65537, 33, 1, None),               # 4: 1025
    (1, 2, 1, 64, 5, 1 << 18, 90, 0, None),             # 4: 4096, 128 KB
    (1, 1, 1, 128, 7, (1 << 18) - 63, 4095, 3, [(1 << 18) - 70]),
]


@pytest.mark.parametrize("B,H,G,D,nq,Sk,keep,first,kv", CASES)
def test_lists(B, H, G, D, nq, Sk, keep, first, kv):
    Sq = nq * 128 - 45
    q, k, v = inputs(B, H, G, D, Sq, Sk, nq + keep)
    kv_len = None if kv is None else torch.tensor(kv, dtype=torch.int32, device=DEV)
    want = lists_64(q, k, kv, keep, first)
    assert torch.equal(bdt.select_blocks(q, k, keep, first, kv_len).cpu(), want)
    q[...] = 1                                                      # many equal scores
    k[...] = (torch.arange(Sk, device=DEV) // 64 % 3).to(torch.bfloat16)[None, None, :, None]
    assert torch.equal(bdt.select_blocks(q, k, keep, first, kv_len).cpu(), lists_64(q, k, kv, keep, first))


def test_attention_after_a_choice_of_16():
    """The whole call where a workgroup chooses for 16 query blocks; some heads compared."""
    q, k, v = inputs(1, 24, 24, 64, 88 * 128 - 45, 1300, 7)
    out, blocks = bdt.sparse_attention(q, k, v, 4, return_blocks=True)
    want = lists_64(q, k, None, 4, 0)
    assert torch.equal(blocks.cpu(), want)
    some = [(0, 0), (0, 23)]
    ref, tol = attention_64(q, k, v, want, 0.125, None, some)
    heads = [h for _, h in some]
    check(out[:, :, heads], ref[:, :, heads], tol[:, :, heads], "heads %s" % heads)

"""Calls that the documentation of paged_attention allows beside the usual ones: queries that are
columns of a projection, pages that several requests share or that a table names twice, a
workspace of the caller's, bit patterns for tensors, calls from two threads."""
import threading

import pytest
import torch

import bit_diffusion_transformer_amd as bdt
from tests import long_keys as lk
from tests.helpers import DEV
from tests.test_gpu_paged_long import ints, starts

pytestmark = pytest.mark.gpu
BF = torch.bfloat16

SETS = [(8, 2, 128, 64, [1, 1, 3], [900, 130, 2000]), (6, 2, 64, 16, [70, 2, 129], [300, 1000, 129]),
        (32, 8, 128, 32, [600, 1, 4], [1700, 3000, 9])]
sets = pytest.mark.parametrize("H,G,D,page,new,lens", SETS)


def made(H, G, D, page, new, lens):
    ks = [lk.normal(10 + b, m, G, D, device=DEV) for b, m in enumerate(lens)]
    vs = [lk.normal(20 + b, m, G, D, device=DEV) for b, m in enumerate(lens)]
    kc, vc, tables = lk.in_pages(ks, vs, page, 5)
    q = lk.normal(1, sum(new), H, D, device=DEV)
    return q, kc, vc, tables.to(DEV), ints(starts(new)), ints(lens)


@sets
def test_queries_that_are_columns_of_a_projection(H, G, D, page, new, lens):
    q, *rest = made(H, G, D, page, new, lens)
    want = bdt.paged_attention(q, *rest, max_new=max(new))
    for before, behind in ((0, 2 * G * D), (G * D, 8), (8, 0)):
        wide = lk.normal(9, sum(new), before + H * D + behind, device=DEV)
        part = wide[:, before:before + H * D].unflatten(1, (H, D))
        part.copy_(q)
        assert not part.is_contiguous()
        assert torch.equal(bdt.paged_attention(part, *rest, max_new=max(new)), want)
    flat = torch.zeros(q.numel() + 4, dtype=BF, device=DEV)[4:].view(q.shape)
    with pytest.raises(RuntimeError, match="aligned"):
        bdt.paged_attention(flat, *rest, max_new=max(new))
    with pytest.raises(RuntimeError, match="stride"):
        wide = torch.zeros(sum(new), H * D + 4, dtype=BF, device=DEV)[:, :H * D].unflatten(1, (H, D))
        bdt.paged_attention(wide, *rest, max_new=max(new))


@sets
def test_shared_pages(H, G, D, page, new, lens):
    """A common beginning in the pages of one request, and a table that names a page twice."""
    q, kc, vc, tables, at, kv = made(H, G, D, page, new, lens)
    n = min(lens) // page                                   # whole pages of the shortest
    tables[:, :n] = tables[0, :n].clone()
    tables[0, 1 if n > 1 else 0] = tables[0, 0].clone()
    own_k, own_v = [], []
    for b, m in enumerate(lens):
        pages = tables[b, :-(-m // page)].long()
        own_k.append(kc[pages].transpose(1, 2).reshape(-1, G, D)[:m])
        own_v.append(vc[pages].transpose(1, 2).reshape(-1, G, D)[:m])
    k2, v2, t2 = lk.in_pages(own_k, own_v, page, 8)
    for most in (max(new), 1, None):
        got = bdt.paged_attention(q, kc, vc, tables, at, kv, max_new=most)
        assert torch.equal(got, bdt.paged_attention(q, k2, v2, t2[:, :tables.shape[1]].to(DEV).contiguous(), at, kv, max_new=most))


@sets
def test_a_workspace_of_the_caller_and_bit_patterns(H, G, D, page, new, lens):
    q, kc, vc, tables, at, kv = made(H, G, D, page, new, lens)
    want = bdt.paged_attention(q, kc, vc, tables, at, kv, max_new=max(new))
    shape = bdt.PagedShape(sum(new), kc.shape[0], H * D, len(new), H, G, D, page, tables.shape[1], max(new), 1)
    need = bdt.svdq_paged_attention_workspace_bytes(shape)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device=DEV)
    for _ in range(2):                                      # what it holds does not matter
        assert torch.equal(bdt.paged_attention(q, kc, vc, tables, at, kv, max_new=max(new), workspace=ws), want)
    small = torch.zeros(16, dtype=torch.uint8, device=DEV)  # too small: another one is taken
    assert torch.equal(bdt.paged_attention(q, kc, vc, tables, at, kv, max_new=max(new), workspace=small), want)
    bits = [t.view(torch.int16) for t in (q, kc, vc)]
    got = bdt.paged_attention(*bits, tables, at, kv, max_new=max(new), out=torch.empty_like(bits[0]))
    assert torch.equal(got.view(BF), want)


def test_calls_from_two_threads():
    args = [made(*s) for s in SETS]
    want = [bdt.paged_attention(*a, max_new=max(s[4])) for a, s in zip(args, SETS)]
    torch.cuda.synchronize()
    wrong = []

    def work(seed):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for i in range(30):
                    j = (i + seed) % len(SETS)
                    got = bdt.paged_attention(*args[j], max_new=max(SETS[j][4]))
                    stream.synchronize()
                    if not torch.equal(got, want[j]):
                        wrong.append(j)
                    try:
                        bdt.paged_attention(*args[j], max_new=max(SETS[j][4]), scale=-1.0)
                        wrong.append("no error")
                    except RuntimeError as e:
                        if "scale" not in str(e):
                            wrong.append(str(e))
        except Exception as e:
            wrong.append(repr(e))
    threads = [threading.Thread(target=work, args=(s,)) for s in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong

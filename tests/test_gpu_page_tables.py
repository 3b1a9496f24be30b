"""Page tables of a step against a plain count on the host: whole numbers, equal."""
import numpy as np
import pytest
import torch

import bit_diffusion_transformer_amd as bdt
from tests.helpers import DEV

pytestmark = pytest.mark.gpu
MAX = 1 << 30


def ints(x):
    return torch.tensor(np.asarray(x, np.int32), device=DEV)


def plain(cached, added, free, tables, page, pages, T):
    """The documented result, token by token of the first T."""
    tables = [list(r) for r in tables]
    width = len(tables[0]) if tables else 0
    starts, kv, slots, positions, taken, lost, at = [], [], [], [], 0, 0, 0
    for b, (c, n) in enumerate(zip(cached, added)):
        c, n = min(max(c, 0), MAX), max(n, 0)
        held = -(-c // page)
        want = max(min(-(-(c + n) // page), width) - held, 0)
        for i in range(want):
            j = taken + i
            tables[b][held + i] = free[j] if j < len(free) else -1
        taken += want
        starts.append(min(at, T))
        kv.append(min(c + n, MAX))
        for p in range(c, c + min(n, max(T - at, 0))):
            entry = tables[b][p // page] if p // page < width else -1
            slots.append(entry * page + p % page if 0 <= entry < pages else -1)
            positions.append(p)
            lost += slots[-1] < 0
        lost += n - min(n, max(T - at, 0))
        at += n
    starts.append(min(at, T))
    slots += [-1] * (T - len(slots))
    positions += [-1] * (T - len(positions))
    return tables, starts, kv, slots, positions, [taken, min(lost, 2 ** 31 - 1)]


def check(cached, added, free, tables, page, pages, T):
    tables = np.asarray(tables, np.int32).reshape(len(cached), -1)
    dev = ints(tables)
    want = plain(cached, added, free, tables.tolist(), page, pages, T)
    for _ in range(2):                               # the same call again gives the same
        got = bdt.page_tables(ints(cached), ints(added), ints(free), dev, page, pages, T)
        for what, x, y in zip(("tables", "q_starts", "kv_len", "slots", "positions", "counts"),
                              (dev,) + got, want):
            assert x.cpu().tolist() == y, what


@pytest.mark.parametrize("B,page,top,more,seed", [
    (1, 16, 1, 1, 0), (1, 256, 700, 3000, 1), (5, 16, 40, 20, 2), (64, 16, 8000, 1, 3),
    (255, 32, 300, 4, 4), (256, 64, 900, 70, 5), (257, 128, 500, 9, 6), (512, 64, 4000, 260, 7),
    (1024, 16, 200, 3, 8), (1025, 16, 60, 5, 9), (8192, 32, 100, 2, 10), (3, 16, 0, 4000, 11),
])
def test_page_tables(B, page, top, more, seed):
    rng = np.random.default_rng(seed)
    cached = np.where(rng.random(B) < 0.3, 0, rng.integers(0, top + 1, B)).tolist()
    added = rng.integers(0, more + 1, B).tolist()
    held = [-(-c // page) for c in cached]
    need = sum(-(-(c + n) // page) - h for c, n, h in zip(cached, added, held))
    pages = sum(held) + need + 7
    order = rng.permutation(pages).tolist()
    width = max(-(-(c + n) // page) for c, n in zip(cached, added)) + int(rng.integers(0, 3))
    tables, at = np.full((B, max(width, 1)), -9), 0
    for b, h in enumerate(held):
        tables[b, :h] = order[at:at + h]
        at += h
    T = sum(added)
    check(cached, added, order[at:], tables, page, pages, T + int(rng.integers(0, 40)))
    check(cached, added, order[at:], tables, page, pages, T)


def test_what_does_not_fit():
    """Free pages that end, a table that is too narrow, more tokens than T, bad entries in the
    table and among the free pages, lengths below zero and past the limit."""
    check([5, 0, 40], [30, 10, 20], [3, 1], [[7, -1, -1], [-1] * 3, [2, 4, 0]], 16, 9, 60)
    check([5, 0, 40], [30, 10, 20], [], [[7, -1, -1], [-1] * 3, [2, 4, 0]], 16, 9, 60)
    check([5, 0, 40], [100, 10, 90], list(range(3, 9)), [[7, -1, -1], [-1] * 3, [2, 4, 0]], 16, 9, 200)
    check([5, 0, 40], [30, 10, 20], list(range(3, 9)), [[7, -1, -1], [-1] * 3, [2, 4, 0]], 16, 9, 33)
    check([5, 0, 40], [30, 10, 20], list(range(3, 9)), [[7, -1, -1], [-1] * 3, [2, 4, 0]], 16, 9, 0)
    check([5, 20, 40], [3, 10, 20], [9, -1, 3, 2 ** 31 - 1, -2 ** 31], [[9, -1, -1], [0, -4, 0], [2, 4, 2 ** 30]],
          16, 9, 60)
    check([-5, 3, -2 ** 31], [5, -1, 7], [1, 2, 3], [[-1], [0], [-1]], 32, 4, 12)
    check([50, 3], [5, 4], [1, 2, 3], [[0], [1]], 32, 4, 12)             # more cached than the table
    check([2 ** 31 - 1, 0], [3, 5], [1, 2], [[0, 1], [1, 0]], 16, 4, 8)
    check([2 ** 30 - 1, 0], [3, 5], [1, 2], [[0, 1], [1, 0]], 16, 4, 8)
    check([0] * 300, [1] * 300, list(range(150)), [[-1]] * 300, 16, 150, 300)


def test_added_past_every_limit():
    cached, added = [1, 2], [2 ** 31 - 1, 2 ** 31 - 1]
    dev = ints([[0, -1, -1], [1, -1, -1]])
    starts, kv, slots, positions, counts = bdt.page_tables(ints(cached), ints(added), ints([5, 6, 7]), dev,
                                                           16, 8, 20)
    assert starts.tolist() == [0, 20, 20] and kv.tolist() == [MAX, MAX]
    assert positions.tolist() == list(range(1, 21))
    assert slots.tolist() == list(range(1, 16)) + [80 + i for i in range(5)]
    assert counts.tolist() == [4, 2 ** 31 - 1]
    assert dev.tolist() == [[0, 5, 6], [1, 7, -1]]


def test_parts_of_larger_arrays():
    """int32 arrays that start at any element."""
    cached, added, free = [5, 0, 40], [30, 10, 20], list(range(3, 9))
    t = [[7, -1, -1], [-1] * 3, [2, 4, 0]]
    want = plain(cached, added, free, t, 16, 9, 60)
    for off in range(4):
        b = ints([0] * off + cached + added + free + sum(t, []))
        x = b[off + 12:off + 21].view(3, 3)
        got = (x,) + bdt.page_tables(b[off:off + 3], b[off + 3:off + 6], b[off + 6:off + 12], x, 16, 9, 60)
        assert [y.tolist() for y in got] == list(want)


def test_no_requests_and_no_tokens():
    none = torch.empty(0, dtype=torch.int32, device=DEV)
    out = bdt.page_tables(none, none, none, none.view(0, 0), 16, 0, 5)
    assert [x.tolist() for x in out] == [[0], [], [-1] * 5, [-1] * 5, [0, 0]]
    out = bdt.page_tables(none, none, none, none.view(0, 4), 16, 9, 0)
    assert [x.tolist() for x in out] == [[0], [], [], [], [0, 0]]
    out = bdt.page_tables(ints([3]), ints([2]), none, none.view(1, 0), 16, 9, 2)
    assert [x.tolist() for x in out] == [[0, 2], [5], [-1, -1], [3, 4], [0, 2]]


def test_replayed_with_other_lengths():
    B, page, pages, width = 40, 16, 600, 12
    rng = np.random.default_rng(0)
    cached, added, free = ints([0] * B), ints([0] * B), ints(rng.permutation(pages))
    tables = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    bdt.page_tables(cached, added, free, tables, page, pages, 900)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = bdt.page_tables(cached, added, free, tables, page, pages, 900)
    for it in range(4):
        c, n = rng.integers(0, 100, B).tolist(), rng.integers(0, 20, B).tolist()
        t = rng.integers(0, pages, (B, width)).tolist()
        for dst, src in ((cached, c), (added, n), (tables, t)):
            dst.copy_(ints(src))
        graph.replay()
        torch.cuda.synchronize()
        want = plain(c, n, free.tolist(), t, page, pages, 900)
        for x, y in zip((tables,) + out, want):
            assert x.cpu().tolist() == y, "replay %d" % it

"""Block tables and slot maps from request lengths, against lists kept on the host."""
import pytest
import torch

from tests import _paged as P
from exact_io_aware_14_gb300 import _native as A

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def state(g, B, blocks, page, lens, num):
    """Tables of sequences that hold lens tokens, and the free list that is left of num pages."""
    pages = torch.randperm(num, generator=g).tolist()
    table = [[-1] * blocks for _ in range(B)]
    for b in range(B):
        for j in range(-(-lens[b] // page)):
            table[b][j] = pages.pop()
    return table, pages + [-7] * (num - len(pages)), len(pages)


def run_reserve(table, lens, new, free, count, page, max_new, slots=True):
    t, so = i32(table), torch.full((len(lens),), -5, dtype=torch.int32, device="cuda")
    granted, sl, c = A.kvcache_reserve_paged(t, i32(lens), None if new is None else i32(new), i32(free), i32([count]),
                                             page, max_new, slots=slots, seqlens_out=so)
    assert A.attn_get_device_status() == 0
    return t.tolist(), granted.tolist(), None if sl is None else sl.tolist(), int(c), so.tolist()


@pytest.mark.parametrize("B,blocks,page,max_new,hi,short", [
    (1, 1, 64, 1, 0, 0), (1, 4, 64, 64, 100, 0), (5, 40, 64, 1, 700, 0), (5, 40, 64, 1, 700, 1), (7, 30, 192, 3000, 900, 0),
    (7, 30, 192, 3000, 900, 3), (300, 5, 256, 300, 700, 0), (300, 5, 256, 300, 700, 5), (1500, 3, 64, 5, 150, 2),
    (2500, 3, 64, 5, 150, 0)])
def test_reserve(B, blocks, page, max_new, hi, short):
    g = torch.Generator().manual_seed(B + max_new)
    lens = torch.randint(0, hi + 1, (B,), generator=g).tolist()
    new = torch.randint(0, max_new + 1, (B,), generator=g).tolist()
    lens = [min(n, blocks * page - m) for n, m in zip(lens, new)]
    need = sum(-(-(n + m) // page) - -(-n // page) for n, m in zip(lens, new))
    used = sum(-(-n // page) for n in lens)
    left = max(0, need - short) if short else need + 3
    table, free, count = state(g, B, blocks, page, lens, used + left)
    want = P.reserve(table, lens, new, free, count, page, max_new)
    got = run_reserve(table, lens, new, free, count, page, max_new)
    assert got[0] == want[0] and got[1] == want[1] and got[2] == want[2] and got[3] == want[3]
    assert got[4] == [n + m for n, m in zip(lens, want[1])]


def test_reserve_without_slots_and_with_equal_requests():
    g = torch.Generator().manual_seed(3)
    lens = [0, 63, 64, 65, 128]
    table, free, count = state(g, 5, 6, 64, lens, 40)
    want = P.reserve(table, lens, [65] * 5, free, count, 64, 65)
    got = run_reserve(table, lens, None, free, count, 64, 65, slots=False)
    assert got[0] == want[0] and got[1] == [65] * 5 and got[2] is None and got[3] == want[3]


def test_a_sequence_with_room_is_served_when_the_pages_ran_out():
    table = [[0, -1, -1], [1, -1, -1], [2, -1, -1], [3, -1, -1]]
    got = run_reserve(table, [60, 64, 10, 64], [4, 65, 50, 1], [9, 8, 7, 6] + [0] * 8, 1, 64, 65)
    # the second wants two pages where one is free; the last one then gets none either
    assert got[1] == [4, 0, 50, 0] and got[3] == 1 and got[0] == table


@pytest.mark.parametrize("B,blocks,page,hi", [(1, 2, 64, 128), (6, 20, 64, 1200), (40, 9, 192, 1700), (2100, 3, 64, 190)])
def test_release(B, blocks, page, hi):
    g = torch.Generator().manual_seed(B)
    lens = torch.randint(0, hi + 1, (B,), generator=g).tolist()
    keep = [int(torch.randint(0, n + 1, (1,), generator=g)) if b % 3 else 0 for b, n in enumerate(lens)]
    table, free, count = state(g, B, blocks, page, lens, sum(-(-n // page) for n in lens) + 2)
    f, t = i32(free), i32(table)
    c = A.kvcache_release_paged(t, i32(lens), i32(keep), f, i32([count]), page)
    assert A.attn_get_device_status() == 0
    want, wc = P.release(table, lens, keep, free, count, page)
    assert f.tolist() == want and int(c) == wc and t.tolist() == table


def test_release_undoes_a_reserve():
    g = torch.Generator().manual_seed(8)
    lens, new = [0, 100, 64, 7], [200, 30, 64, 50]
    table, free, count = state(g, 4, 5, 64, lens, 30)
    t, f = i32(table), i32(free)
    granted, _, c = A.kvcache_reserve_paged(t, i32(lens), i32(new), f, i32([count]), 64, 200)
    after = i32(lens) + granted
    c = A.kvcache_release_paged(t, after, i32(lens), f, c, 64)
    assert f.tolist() == free and int(c) == count


@pytest.mark.parametrize("lens,new,granted", [([-1, 10], [5, 5], [0, 5]), ([10, 10], [6, 5], [0, 5]),
                                              ([190, 10], [5, 5], [0, 5]), ([10, 500], [5, 5], [5, 0]),
                                              ([10, 10], [-2, 5], [0, 5])])
def test_reserve_reports_lengths_out_of_range(lens, new, granted):
    t = i32([[0, 1, 2], [3, -1, -1]])
    got, sl, c = A.kvcache_reserve_paged(t, i32(lens), i32(new), i32([9, 8, 7, 6] + [0] * 8), i32([4]), 64, 5)
    assert A.attn_get_device_status() == A.ATTN_ERR_DEVICE_ARG
    assert got.tolist() == granted and t.tolist() == [[0, 1, 2], [3, -1, -1]] and int(c) == 4


@pytest.mark.parametrize("count", [-1, 13])
def test_a_bad_count_is_reported(count):
    A.kvcache_reserve_paged(i32([[0, 1, 2]]), i32([10]), i32([1]), i32([9] * 12), i32([count]), 64, 1)
    assert A.attn_get_device_status() == A.ATTN_ERR_DEVICE_ARG


def test_release_reports_bad_lengths_and_too_many_pages():
    f = i32([5, 6, 7])
    c = A.kvcache_release_paged(i32([[0, 1, 2]]), i32([100]), i32([101]), f, i32([2]), 64)
    assert A.attn_get_device_status() == A.ATTN_ERR_DEVICE_ARG and int(c) == 2 and f.tolist() == [5, 6, 7]
    c = A.kvcache_release_paged(i32([[0, 1, 2]]), i32([100]), i32([0]), f, i32([2]), 64)
    assert A.attn_get_device_status() == A.ATTN_ERR_DEVICE_ARG and int(c) == 3 and f.tolist() == [5, 6, 1]


def test_a_captured_step_follows_its_lengths():
    g = torch.Generator().manual_seed(1)
    lens = [10, 64, 130]
    table, free, count = state(g, 3, 8, 64, lens, 20)
    t, l, f, c, n = i32(table), i32(lens), i32(free), i32([count]), i32([60, 60, 60])
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        A.kvcache_reserve_paged(t.clone(), l, n, f, c, 64, 60)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        granted, slots, c2 = A.kvcache_reserve_paged(t, l, n, f, c, 64, 60)
        l.add_(granted)
        c.copy_(c2)
    for step in range(3):
        graph.replay()
        table, want, sl, count = P.reserve(table, lens, [60] * 3, free, count, 64, 60)
        lens = [a + b for a, b in zip(lens, want)]
        torch.cuda.synchronize()
        assert t.tolist() == table and granted.tolist() == want and slots.tolist() == sl and int(c) == count
        assert l.tolist() == lens
    assert A.attn_get_device_status() == 0

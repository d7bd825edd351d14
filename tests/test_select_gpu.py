"""Key bounds and block selection, against their definitions on the host."""
import pytest
import torch

from tests import _paged as P
from exact_io_aware_14_gb300 import _native as A

pytestmark = pytest.mark.gpu


def dev(*t):
    return [x.cuda() for x in t]


@pytest.mark.parametrize("B,Hkv,d,page,lens,new", [
    (1, 1, 64, 64, [1], [1]), (1, 1, 128, 64, [64], [64]), (3, 2, 128, 64, [65, 63, 200], [1, 63, 137]),
    (4, 5, 64, 192, [500, 1, 192, 0], [400, 1, 0, 0]), (2, 8, 128, 256, [700, 513], [513, 512]), (2, 9, 128, 128, [300, 129], [2, 129])])
def test_bounds(B, Hkv, d, page, lens, new):
    g = torch.Generator().manual_seed(len(lens) * d + Hkv)
    table, num = P.tables(g, B, -(-max(lens) // page) + 1, 0)
    kp, = P.pools(g, num, page, Hkv, d, 1)
    kb = torch.randn((num, page // 64, Hkv, 2, d), generator=g).to(torch.bfloat16)
    for b, L in enumerate(lens):  # behind the end: of no meaning
        kp[table[b, L // page].long(), L % page:] = float("nan")
    want = P.bounds(kp, table, page, lens, new, kb)
    k, b, t = dev(kp, kb, table)
    A.kvcache_bounds_paged(k, b, t, torch.tensor(lens, dtype=torch.int32).cuda(), max(new),
                           torch.tensor(new, dtype=torch.int32).cuda())
    assert A.attn_get_device_status() == 0
    assert torch.equal(b.cpu(), want)
    assert torch.equal(k.cpu().view(torch.int16), kp.view(torch.int16))


def test_bounds_of_equal_counts_whole_sequences_and_bad_lengths():
    g = torch.Generator().manual_seed(5)
    table, num = P.tables(g, 3, 4, 0)
    kp, = P.pools(g, num, 64, 2, 64, 1)
    kp[table[1, 0].long(), 3, 1, 7] = float("nan")
    kp[table[1, 0].long(), 4, 1, 8] = float("inf")
    lens = [250, 70, 5]
    kb = torch.zeros((num, 1, 2, 2, 64), dtype=torch.bfloat16)
    want = P.bounds(kp, table, 64, lens, [100, 70, 5], kb)
    k, b, t = dev(kp, kb, table)
    A.kvcache_bounds_paged(k, b, t, torch.tensor(lens, dtype=torch.int32).cuda(), 100)
    assert A.attn_get_device_status() == 0
    assert torch.equal(b.cpu().isnan(), want.isnan()) and int(want.isnan().sum()) == 2
    assert torch.equal(b.cpu().nan_to_num(), want.nan_to_num())
    A.kvcache_bounds_paged(k, b, t, torch.tensor([257, 0, 1], dtype=torch.int32).cuda(), 1)
    assert A.attn_get_device_status() == A.ATTN_ERR_DEVICE_ARG
    t[2, 0] = num
    A.kvcache_bounds_paged(k, b, t, torch.tensor(lens, dtype=torch.int32).cuda(), 1)
    assert A.attn_get_device_status() == A.ATTN_ERR_DEVICE_ARG


def case(seed, B, Nq, Hq, Hkv, d, page, blocks):
    g = torch.Generator().manual_seed(seed)
    table, num = P.tables(g, B, blocks, 0)
    kp, = P.pools(g, num, page, Hkv, d, 1)
    x = kp.view(num, page // 64, 64, Hkv, d)
    kb = torch.stack((x.amin(2), x.amax(2)), 3)
    return torch.randn((B, Nq, Hq, d), generator=g).to(torch.bfloat16), kb, table


def run(q, kb, table, lens, topk, sink=1, local=1):
    q, kb, t = dev(q, kb, table)
    out = A.select_blocks_paged(q, kb, t, torch.tensor(lens, dtype=torch.int32).cuda(), topk, sink, local)
    assert A.attn_get_device_status() == 0
    return out.cpu()


@pytest.mark.parametrize("B,Nq,Hq,Hkv,d,page,lens,topk,sink,local", [
    (1, 1, 1, 1, 64, 64, [1], 1, 0, 0), (1, 1, 1, 1, 64, 64, [1], 4, 1, 1), (2, 1, 4, 2, 128, 64, [64, 1000], 5, 1, 1),
    (3, 3, 9, 3, 64, 192, [2, 700, 3000], 7, 0, 0), (2, 1, 8, 1, 128, 256, [5000, 4097], 1, 0, 0),
    (2, 70, 10, 2, 128, 64, [75, 2000], 6, 2, 2), (1, 1, 128, 1, 128, 128, [9000], 100, 3, 5), (1, 200, 4, 4, 64, 64, [200], 3, 1, 1),
    (1, 2, 4, 2, 64, 64, [70000], 64, 1, 2), (2, 1, 2, 2, 64, 64, [900, 0], 2, 1, 1), (1, 1, 7, 1, 64, 64, [2100], 16, 16, 0),
    # up to 16, up to 64 and more rows of a sequence
    (1, 16, 1, 1, 64, 64, [9000], 9, 1, 1), (1, 17, 1, 1, 128, 64, [9000], 9, 1, 1), (2, 16, 8, 2, 128, 64, [3000, 9], 5, 1, 1),
    (3, 3, 10, 1, 64, 192, [700, 20000, 2], 7, 0, 1), (1, 1, 64, 1, 128, 128, [5000], 6, 1, 0), (1, 5, 13, 1, 64, 64, [9000], 8, 1, 1),
    # more tokens than blocks, and fewer
    (1, 330, 1, 1, 64, 64, [20100], 9, 1, 1), (1, 300, 1, 1, 64, 64, [20100], 9, 1, 1), (1, 650, 1, 1, 64, 64, [40000], 12, 2, 1),
    (1, 1110, 1, 1, 64, 64, [70000], 16, 1, 3), (1, 900, 1, 1, 64, 64, [70000], 16, 1, 3)])
def test_selection(B, Nq, Hq, Hkv, d, page, lens, topk, sink, local):
    q, kb, table = case(Nq + Hq + topk, B, Nq, Hq, Hkv, d, page, -(-max(lens) // page))
    assert torch.equal(run(q, kb, table, lens, topk, sink, local),
                       P.select(q, kb, table, page, lens, topk, sink, local))


@pytest.mark.parametrize("n", [20, 700, 1100, 2600])
def test_equal_scores_take_the_lower_index(n):
    q, kb, table = case(n, 1, 2, 2, 1, 64, 64, n)
    kb[:] = kb[:1]  # every block the same
    got = run(q, kb, table, [64 * n], 9, 1, 2)
    assert torch.equal(got, P.select(q, kb, table, 64, [64 * n], 9, 1, 2))
    assert got[0, 1, 0].tolist() == [0, 1, 2, 3, 4, 5, 6, n - 2, n - 1]
    # some of a few kinds
    q, kb, table = case(n, 1, 2, 2, 1, 64, 64, n)
    kb = kb[torch.arange(len(kb)) % 5]
    assert torch.equal(run(q, kb, table, [64 * n], n // 3, 0, 1), P.select(q, kb, table, 64, [64 * n], n // 3, 0, 1))


def test_scores_that_differ_in_their_last_bits():
    # products of very different sizes: a sum in 32 bits loses the small ones, which alone tell the blocks apart
    n = 40
    q, kb, table = case(9, 1, 1, 2, 1, 128, 64, n)
    g = torch.Generator().manual_seed(2)
    q[:] = 1
    kb[:] = 0
    kb[:, 0, 0, :, 0], kb[:, 0, 0, :, 1] = 2.0 ** 14, -(2.0 ** 14)
    kb[:, 0, 0, :, 5] = ((torch.randperm(len(kb), generator=g)[:, None] - 20) * 2.0 ** -14).to(torch.bfloat16)
    got = run(q, kb, table, [64 * n], 10, 0, 0)
    assert torch.equal(got, P.select(q, kb, table, 64, [64 * n], 10, 0, 0))


@pytest.mark.parametrize("what", ["nan key", "inf key", "nan query", "zero query", "inf query"])
def test_values_that_are_not_numbers_and_zeros(what):
    n = 30
    q, kb, table = case(4, 1, 1, 4, 2, 64, 64, n)
    if what == "nan key":
        kb[table[0, 7].long(), 0, 0, :, 3] = float("nan")
    elif what == "inf key":
        kb[table[0, 7].long(), 0, 1, 1, 3] = float("inf")
    elif what == "nan query":
        q[0, 0, 1, 5] = float("nan")
    elif what == "inf query":
        q[0, 0, 1, 5] = float("inf")
    else:
        q[:] = 0
    got = run(q, kb, table, [64 * n], 6)
    assert torch.equal(got, P.select(q, kb, table, 64, [64 * n], 6, 1, 1))
    if what.endswith("key"):
        assert 7 in got[0, 0, 0 if what == "nan key" else 1].tolist()


@pytest.mark.parametrize("n", [300, 1500, 2500])
def test_a_padded_token_takes_the_lowest_blocks(n):
    q, kb, table = case(n, 1, 2, 4, 1, 64, 64, n)
    q[0, 0] = 0
    q[0, 0, 1, 3] = -0.0
    got = run(q, kb, table, [64 * n], 12, 1, 2)
    assert torch.equal(got, P.select(q, kb, table, 64, [64 * n], 12, 1, 2))
    assert got[0, 0, 0].tolist() == list(range(10)) + [n - 2, n - 1]


def test_products_outside_the_range_of_32_bits():
    n = 24
    for size in (2.0 ** 100, 2.0 ** -100):
        q, kb, table = case(6, 1, 1, 2, 1, 64, 64, n)
        q, kb = (q.float() * size).to(torch.bfloat16), (kb.float() * size).to(torch.bfloat16)
        assert torch.equal(run(q, kb, table, [64 * n], 6), P.select(q, kb, table, 64, [64 * n], 6, 1, 1))


def test_bad_lengths_and_pages_are_reported():
    q, kb, table = case(1, 1, 1, 2, 1, 64, 64, 8)
    q, kb, t = dev(q, kb, table)
    out = A.select_blocks_paged(q, kb, t, torch.tensor([513], dtype=torch.int32).cuda(), 3)
    assert A.attn_get_device_status() == A.ATTN_ERR_DEVICE_ARG
    assert int(out.max()) < 8 and int(out.min()) >= 0
    t[0, 2] = -1
    A.select_blocks_paged(q, kb, t, torch.tensor([512], dtype=torch.int32).cuda(), 3)
    assert A.attn_get_device_status() == A.ATTN_ERR_DEVICE_ARG


def test_many_tokens_pass_through_a_small_workspace_in_parts():
    # a table so wide that a launch takes few tokens
    q, kb, table = case(12, 1, 9, 2, 2, 64, 64, 20)
    wide = torch.full((1, 1 << 22), -1, dtype=torch.int32)
    wide[:, :20] = table
    got = run(q, kb, wide, [64 * 20], 4)
    assert torch.equal(got, P.select(q, kb, table, 64, [64 * 20], 4, 1, 1))

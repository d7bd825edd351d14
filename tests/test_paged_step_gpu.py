"""A serving step over a paged bf16 cache in which the sequences' new tokens differ in number, against 64 bits, and one with
a bad page in its table."""
import pytest
import torch

from tests import _paged as P
from tests.test_rows_gpu import i32, listed
from exact_io_aware_14_gb300 import _native as A

pytestmark = pytest.mark.gpu


def test_a_step_of_sequences_with_different_counts_of_new_tokens():
    """The append takes the first granted[b] rows, the attention calls take the last tokens of each sequence: the queries
    are moved to the end of their rows.  Each query must meet its own key."""
    g = torch.Generator().manual_seed(41)
    B, n, Hq, Hkv, d, page, num = 4, 5, 8, 2, 64, 64, 40
    kp, vp = (torch.zeros((num, page, Hkv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    kb = torch.zeros((num, 1, Hkv, 2, d), dtype=torch.bfloat16, device="cuda")
    table = torch.full((B, 9), -1, dtype=torch.int32, device="cuda")
    free, count = torch.randperm(num, generator=g).to(torch.int32).cuda(), i32([6])
    lens = i32([0] * B)
    for wanted in ([60, 130, 5, 62], [5, 3, 1, 4], [2, 0, 5, 5]):  # the pages run out in the last two steps
        n = max(wanted)
        k, v, q = (torch.randn((B, n, h, d), generator=g).to(torch.bfloat16).cuda() for h in (Hkv, Hkv, Hq))
        granted, _, count = A.kvcache_reserve_paged(table, lens, i32(wanted), free, count, page, n)
        after = torch.empty_like(lens)
        A.kvcache_append_paged(k, v, kp, vp, table, lens, new_lens=granted, seqlens_out=after)
        A.kvcache_bounds_paged(kp, kb, table, after, n, new_lens=granted)
        row = (torch.arange(n, device="cuda") - (n - granted)[:, None]).clamp_(min=0)
        q_last = q.gather(1, row[..., None, None].expand_as(q))
        blocks = A.select_blocks_paged(q_last, kb, table, after, 3, 1, 1)
        sparse = A.attend_blocks_paged(q_last, kp, vp, table, after, blocks, d ** -0.5)
        dense = A.decode_paged_shared(q_last, kp, vp, table, after, 0, d ** -0.5)
        assert A.attn_get_device_status() == 0
        got, before, new = granted.tolist(), lens.tolist(), after.tolist()
        assert [b + m for b, m in zip(before, got)] == new
        host = [x.cpu() for x in (kp, vp, table)]
        for b in range(B):
            m = got[b]
            if m == 0:
                continue
            one = lambda x, b=b, m=m: (x[0][b:b + 1, n - m:], x[1][b:b + 1, :, n - m:])
            qb, tb = q[b:b + 1, :m].cpu(), host[2][b:b + 1]  # the new tokens' own rows, as they were appended
            assert torch.equal(host[0][tb[0].long()].reshape(-1, Hkv, d)[before[b]:new[b]], k[b, :m].cpu())
            at = lambda _, i, h, b=b: list(range(before[b] + i + 1))
            P.check(*one(dense), P.attend(qb, host[0], host[1], tb, page, d ** -0.5, at))
            chosen = blocks[b:b + 1, n - m:].cpu()
            assert torch.equal(chosen, P.select(qb, kb.cpu(), tb, page, [new[b]], 3, 1, 1))
            P.check(*one(sparse), P.attend(qb, host[0], host[1], tb, page, d ** -0.5, listed(chosen, [new[b]], m)))
        lens = after


def test_a_bad_page_that_is_released_is_reported_again_by_the_reserve_that_takes_it():
    table, free = i32([[3, 99, 5], [6, -1, -1]]), i32([0, 1, 2, -7, -7, -7, -7, -7])
    count = A.kvcache_release_paged(table, i32([192, 64]), i32([0, 0]), free, i32([3]), 64)
    assert A.attn_get_device_status() == A.ATTN_ERR_DEVICE_ARG
    assert int(count) == 7 and free.tolist() == [0, 1, 2, 6, 5, 99, 3, -7]
    fresh = i32([[-1, -1, -1]])
    granted, slots, count = A.kvcache_reserve_paged(fresh, i32([0]), i32([64]), free, count, 64, 64)
    assert A.attn_get_device_status() == 0 and int(count) == 6 and fresh.tolist() == [[3, -1, -1]]
    granted, slots, count = A.kvcache_reserve_paged(fresh, i32([64]), i32([64]), free, count, 64, 64)
    assert A.attn_get_device_status() == A.ATTN_ERR_DEVICE_ARG
    assert int(count) == 5 and slots.tolist() == [[-1] * 64]  # no row of the pools is named for its tokens

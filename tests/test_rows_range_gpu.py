"""Attention of query rows over a paged bf16 cache where scores rise along the keys and values are large, against 64 bits."""
import pytest
import torch

from tests import _paged as P
from tests.test_rows_gpu import by_block, i32, listed, make, random_blocks, run_shared, seen
from exact_io_aware_14_gb300 import _native as A

pytestmark = pytest.mark.gpu


def rising(seed, B, Nq, Hq, Hkv, d, lens, steps, size):
    """Scores (scale 1) that are steps[j % len(steps)] for the keys of 128-key tile j and a little apart within it, values
    of the given size.  The scores are exact: one channel of q is 1, of the keys a number of 8 bits."""
    q, kp, vp, table = make(seed, B, Nq, Hq, Hkv, d, 64, 0, lens, stale=False)
    q[:] = 0
    q[..., 3] = 1
    kp[:] = 0
    for b in range(B):
        n = torch.arange(lens[b])
        at = torch.tensor(steps)[n // 128 % len(steps)] + (n % 5) / 4
        kp[table[b].long()[n // 64], n % 64, :, 3] = at[:, None].to(torch.bfloat16)
    return q, kp, vp * size, table


STEPS = {"rising": [0., 18., 36., 54.], "in steps below 2^96": [-30., 30.], "up and down": [10., -40., 20., -60., 5.], "one step": [0., 12.]}


# rows in the MMA's N (up to 4, 8, 16, 32), and in its M; sizes of the values up to the documented 2^80
@pytest.mark.parametrize("size", [2.0 ** 40, -(2.0 ** 80)])
@pytest.mark.parametrize("steps", list(STEPS))
@pytest.mark.parametrize("B,Nq,Hq,Hkv,d", [(40, 1, 4, 2, 128), (80, 1, 7, 1, 64), (80, 1, 13, 1, 128), (80, 2, 16, 1, 64),
                                            (80, 1, 25, 1, 128), (80, 2, 40, 1, 128)])
def test_large_values_behind_scores_that_rise(B, Nq, Hq, Hkv, d, steps, size):
    # more tiles than CTAs have lanes: each takes several of a sequence's, one after the other
    lens = [1300 + 61 * (i % 13) for i in range(B)]
    q, kp, vp, table = rising(1, B, Nq, Hq, Hkv, d, lens, STEPS[steps], size)
    want = P.attend(q, kp, vp, table, 64, 1.0, seen(lens, Nq))
    assert want[0].isfinite().all()
    P.check(*run_shared(q, kp, vp, table, lens, 0, 1.0), want)
    blocks = torch.arange(32, dtype=torch.int32).expand(B, Nq, Hkv, 32).contiguous()
    o, lse = A.attend_blocks_paged(*(x.cuda() for x in (q, kp, vp, table)), i32(lens), blocks.cuda(), 1.0)
    assert A.attn_get_device_status() == 0
    P.check(o, lse, want)


@pytest.mark.parametrize("size", [1.0, 2.0 ** 80])
def test_large_values_on_a_shared_prefix_and_in_a_prompts_lists(size):
    # prefixes of one tile of rows and of several, long enough that a lane takes several key tiles
    for B, Hq in ((2, 4), (40, 8)):
        shared = 64 * 1280
        lens = [shared + 100 + 50 * i for i in range(B)]
        q, kp, vp, table = rising(2, 1, 1, Hq, 1, 64, [max(lens)], STEPS["rising"], size)
        table = table.expand(B, -1).contiguous()
        q = q.expand(B, -1, -1, -1).contiguous()
        P.check(*run_shared(q, kp, vp, table, lens, shared, 1.0), P.attend(q, kp, vp, table, 64, 1.0, seen(lens, 1)))
    lens, Nq = [1300], 850
    assert by_block(Nq, 4, 1, 64, 40, 21 * 64)
    q, kp, vp, table = rising(3, 1, Nq, 4, 1, 64, lens, STEPS["rising"], size)
    blocks = random_blocks(torch.Generator().manual_seed(4), 1, Nq, 1, 40, lens)
    o, lse = A.attend_blocks_paged(*(x.cuda() for x in (q, kp, vp, table)), i32(lens), blocks.cuda(), 1.0)
    assert A.attn_get_device_status() == 0
    P.check(o, lse, P.attend(q, kp, vp, table, 64, 1.0, listed(blocks, lens, Nq)))

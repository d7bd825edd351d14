"""Attention over listed blocks with 9 to 32 heads a group, against 64 bits."""
import pytest
import torch

from tests import _paged as P
from tests.test_rows_gpu import i32, listed, make, random_blocks
from exact_io_aware_14_gb300 import _native as A

pytestmark = pytest.mark.gpu


# 9 to 32 heads a group on listed blocks: the forms of 16 and of 32 rows; units that one CTA takes whole, and cut ones
@pytest.mark.parametrize("B,Nq,Hq,Hkv,d,page,lens,n_sel", [
    (1, 1, 9, 1, 64, 64, [700], 6), (1, 1, 16, 1, 128, 128, [5000], 40), (2, 3, 24, 2, 64, 64, [900, 3], 7),
    (3, 2, 32, 2, 128, 64, [1, 0, 1500], 9), (1, 1, 17, 1, 128, 256, [9000], 70), (1, 1, 32, 1, 64, 192, [9000], 70),
    (2, 100, 32, 2, 128, 64, [150, 1111], 5), (1, 90, 24, 1, 64, 64, [800], 5), (1, 170, 20, 1, 128, 64, [800], 4),
    (1, 400, 31, 1, 64, 64, [500], 3)])
def test_listed_blocks_of_larger_groups(B, Nq, Hq, Hkv, d, page, lens, n_sel):
    q, kp, vp, table = make(B + Nq + n_sel + Hq, B, Nq, Hq, Hkv, d, page, 0, lens)
    blocks = random_blocks(torch.Generator().manual_seed(n_sel), B, Nq, Hkv, n_sel, lens)
    o, lse = A.attend_blocks_paged(*(x.cuda() for x in (q, kp, vp, table)), i32(lens), blocks.cuda(), d ** -0.5)
    assert A.attn_get_device_status() == 0
    P.check(o, lse, P.attend(q, kp, vp, table, page, d ** -0.5, listed(blocks, lens, Nq)))


@pytest.mark.parametrize("G", [12, 28])
def test_lists_of_larger_groups_as_a_program_may_write_them(G):
    lens, Nq = [460], 20
    q, kp, vp, table = make(30 + G, 1, Nq, 2 * G, 2, 128, 64, 0, lens)
    # any order, blocks twice, passed over, behind the token, lists of nothing
    blocks = torch.randint(-2, 8, (1, Nq, 2, 9), generator=torch.Generator().manual_seed(G), dtype=torch.int32)
    blocks[0, 3] = -1
    o, lse = A.attend_blocks_paged(*(x.cuda() for x in (q, kp, vp, table)), i32(lens), blocks.cuda(), 0.1)
    assert A.attn_get_device_status() == 0
    P.check(o, lse, P.attend(q, kp, vp, table, 64, 0.1, listed(blocks, lens, Nq)))

"""Block selection where its scores are hard to tell apart in 32 bits, against the definition in 64 bits on the host.
The scores here are exact in double precision, so the order has one answer."""
import pytest
import torch

from tests import _paged as P
from tests.test_select_gpu import case, run

pytestmark = pytest.mark.gpu


def near_ties(n, Nq, Hq, Hkv, d, side, power, seed=0):
    """Blocks whose scores are the same sum in different orders: 8-bit numbers from 1 down to 2^-36, so the sums fit 53
    bits, while sums in 32 bits differ.  One side is scaled by 2^power."""
    q, kb, table = case(seed, 1, Nq, Hq, Hkv, d, 64, n)
    g = torch.Generator().manual_seed(seed + 1)
    x = torch.randint(128, 256, (d,), generator=g).double() * 2.0 ** (-7 - torch.randint(0, 30, (d,), generator=g).double())
    for j in range(n):
        for h in range(Hkv):
            kb[table[0, j].long(), 0, h] = x[torch.randperm(d, generator=g)].to(torch.bfloat16)
    q[:] = 1
    if side == "q":
        q *= 2.0 ** power
    else:
        kb *= 2.0 ** power
    return q, kb, table


@pytest.mark.parametrize("side", ["q", "bounds"])
@pytest.mark.parametrize("power", [0, -60, -74, -76, -90, -96])
@pytest.mark.parametrize("n,Nq,Hq,Hkv,d", [(64, 1, 1, 1, 128), (64, 6, 4, 2, 64), (64, 80, 2, 1, 64), (70, 40, 2, 2, 128),
                                           (2200, 1, 2, 1, 64)])
def test_equal_scores_of_small_queries_or_small_bounds(side, power, n, Nq, Hq, Hkv, d):
    q, kb, table = near_ties(n, Nq, Hq, Hkv, d, side, power)
    got = run(q, kb, table, [64 * n], 9, 0, 0)
    want = P.select(q, kb, table, 64, [64 * n], 9, 0, 0)
    assert want[0, Nq - 1, 0].tolist() == list(range(9))
    assert torch.equal(got, want)


@pytest.mark.parametrize("power", [-76, -100, -133])
def test_one_head_and_one_block_that_are_not_small(power):
    # the largest norms, not the smallest, bound the error
    q, kb, table = near_ties(64, 3, 4, 1, 128, "q", power)
    q[0, 1, 2] = 1
    kb[table[0, 20].long()] = 2
    assert torch.equal(run(q, kb, table, [64 * 64], 9, 1, 1), P.select(q, kb, table, 64, [64 * 64], 9, 1, 1))
    q, kb, table = near_ties(64, 3, 4, 1, 128, "bounds", power)
    kb[table[0, 20].long()] = 2
    assert torch.equal(run(q, kb, table, [64 * 64], 9, 1, 1), P.select(q, kb, table, 64, [64 * 64], 9, 1, 1))


@pytest.mark.parametrize("power", [-80, -133, -200])
def test_a_padded_token_beside_small_bounds(power):
    q, kb, table = near_ties(300, 2, 2, 1, 64, "bounds", power)
    q[0, 0] = 0
    got = run(q, kb, table, [64 * 300], 9, 1, 1)
    assert torch.equal(got, P.select(q, kb, table, 64, [64 * 300], 9, 1, 1))
    assert got[0, 0, 0].tolist() == list(range(8)) + [299]


@pytest.mark.parametrize("d,Nq", [(128, 1), (128, 70), (64, 1), (64, 70)])
def test_scores_that_two_32_bit_numbers_do_not_tell_apart(d, Nq):
    # 1 + 1.5 2^-25 and, for one block, many numbers of 2^-50, each less than half of what the second of two 32-bit
    # numbers (2^-25 and up) resolves; for the other one number of 2^-48 that it does resolve.
    n = 40
    q, kb, table = case(3, 1, Nq, 1, 1, d, 64, n)
    q[:] = 1
    kb[:] = 0
    many, one = torch.zeros(d), torch.zeros(d)
    at = [i for i in range(d) if i % 64 < 8]
    many[at] = 2.0 ** -50  # 6 or 14 of them stay: above 2^-48
    many[0] = one[0] = 1
    many[1] = one[1] = 1.5 * 2.0 ** -25
    one[2] = 2.0 ** -48
    kb[table[0, 9].long(), 0, 0] = many.to(torch.bfloat16)
    kb[table[0, 4].long(), 0, 0] = one.to(torch.bfloat16)
    want = P.select(q, kb, table, 64, [64 * n], 1, 0, 0)
    assert want.flatten().tolist() == [9] * Nq
    assert torch.equal(run(q, kb, table, [64 * n], 1, 0, 0), want)


@pytest.mark.parametrize("Nq", [1, 60])
def test_scores_of_products_that_32_bits_do_not_hold_beside_ordinary_norms(Nq):
    n = 40
    q, kb, table = case(5, 1, Nq, 1, 1, 64, 64, n)
    g = torch.Generator().manual_seed(6)
    q[:] = 0
    q[..., 0], q[..., 1] = 1, 2.0 ** -72
    kb[:] = 0
    kb[:, 0, 0, :, 2] = 1  # the norms' part, which q does not meet
    kb[:, 0, 0, :, 1] = ((128 + torch.randperm(len(kb), generator=g)) * 2.0 ** -79)[:, None].to(torch.bfloat16)
    want = P.select(q, kb, table, 64, [64 * n], 9, 0, 0)
    assert want[0, 0, 0].tolist() != list(range(9))
    assert torch.equal(run(q, kb, table, [64 * n], 9, 0, 0), want)

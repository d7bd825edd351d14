"""Block selection over more blocks than a CTA keeps the scores of, and for many tokens with groups of every size that is
read in its own way, against the definition in 64 bits on the host."""
import pytest
import torch

from tests import _paged as P
from tests.test_select_gpu import case, run

pytestmark = pytest.mark.gpu


def many_blocks(kind, n, Nq, seed=0):
    q, kb, table = case(seed, 1, Nq, 2, 1, 64, 64, n)
    if kind == "equal":
        kb[:] = kb[:1]
    elif kind == "few kinds":
        kb = kb[torch.arange(len(kb)) % 7]
    elif kind == "equal on top":  # fewer than are scored again one by one
        top = 3 * kb.float().abs().amax((0, 1, 2, 3)).to(torch.bfloat16)
        at = table[0, torch.randperm(n, generator=torch.Generator().manual_seed(1))[:60]].long()
        kb[at, 0, 0, 0], kb[at, 0, 0, 1] = -top, top
    elif kind == "zero query":
        q[0, -1] = 0
    elif kind == "nan":
        kb[table[0, n // 2].long(), 0, 0, 1, 5] = float("nan")
    return q, kb, table


# more blocks than a CTA keeps the scores of (8192), and as many, with more to be put in order
@pytest.mark.parametrize("kind", ["random", "equal", "few kinds", "equal on top", "zero query", "nan"])
@pytest.mark.parametrize("n,topk,sink,local", [(8300, 40, 1, 2), (9001, 33, 0, 0), (8197, 21, 4, 3), (8197, 7, 4, 3), (8193, 5, 5, 0)])
def test_more_blocks_than_are_kept(kind, n, topk, sink, local):
    q, kb, table = many_blocks(kind, n, 2)
    assert torch.equal(run(q, kb, table, [64 * n - 5], topk, sink, local),
                       P.select(q, kb, table, 64, [64 * n - 5], topk, sink, local))


@pytest.mark.parametrize("Nq", [131, 129, 257])
@pytest.mark.parametrize("G,d", [(1, 128), (2, 64), (3, 128), (4, 64), (5, 128), (8, 64), (9, 64)])
def test_many_tokens_of_small_and_larger_groups(G, d, Nq):
    q, kb, table = case(G + Nq, 1, Nq, 2 * G, 2, d, 64, 70)
    assert torch.equal(run(q, kb, table, [4400], 6, 1, 1), P.select(q, kb, table, 64, [4400], 6, 1, 1))

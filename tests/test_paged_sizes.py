"""Workspaces of the operators on a paged cache: one buffer for calls of several sizes (no GPU)."""
import pytest

from tests.test_paged_abi import L, attend, select  # noqa: F401


@pytest.mark.parametrize("Nq,n_sel", [(2048, 32), (600, 16)])
def test_a_list_attention_buffer_of_the_widest_table_may_not_do_for_a_narrower_one(L, Nq, n_sel):  # noqa: F811
    size = lambda keys: L.attn_fwd_blocks_paged_workspace_size(1, Nq, 32, 8, 128, n_sel, keys)
    widths = [1 << n for n in range(10, 21)]
    assert size(widths[-1]) < 1 << 24 < size(widths[0])
    # each width takes its own size and refuses less; the largest of them does for all
    args = dict(B=1, Nq=Nq, Hq=32, Hkv=8, d=128, n=n_sel, ps=64, np=1 << 14, o=1 << 40, kp=1 << 36, vp=1 << 37)
    for w in widths:
        assert attend(L, True, mb=w // 64, wsb=size(w) - 1, **args) == 7
        assert attend(L, True, mb=w // 64, wsb=max(map(size, widths)), ws=8, **args) == 7
    assert attend(L, True, mb=widths[0] // 64, wsb=size(widths[-1]), **args) == 7


def test_a_selection_buffer_is_of_the_tables_width(L):  # noqa: F811
    for keys in (64, 1024, 8192, 1 << 17, 1 << 20):
        n = L.attn_select_blocks_workspace_size(4, 300, 2, keys)
        assert n > 0 and select(L, Nq=300, mb=keys // 64, ps=64, wsb=n - 1) == 7

"""Host-side argument checks of the operators on a paged cache (no GPU: every C
call here returns before any CUDA call), and the definitions that the GPU tests
compare with."""
import ctypes
import math

import pytest
import torch

from tests import _paged as P
from exact_io_aware_14_gb300 import _native as A, build as native_build


@pytest.fixture(scope="module")
def L():
    native_build.build()
    return A.lib()


def vp(x):
    return ctypes.c_void_p(x) if x else None


M = 1 << 20  # tensors a MiB apart


def reserve(L, **kw):
    a = dict(bt=M, mb=8, ps=64, np=40, sl=2 * M, nl=3 * M, fp=4 * M, fc=5 * M, no=6 * M, so=7 * M, sm=8 * M, co=9 * M, B=4,
             Nn=5)
    a.update(kw)
    return L.attn_kvcache_reserve_paged(vp(a["bt"]), a["mb"], a["ps"], a["np"], vp(a["sl"]), vp(a["nl"]), vp(a["fp"]),
                                        vp(a["fc"]), vp(a["no"]), vp(a["so"]), vp(a["sm"]), vp(a["co"]), a["B"], a["Nn"],
                                        None)


@pytest.mark.parametrize("want,kw", [
    (1, dict(B=0)), (1, dict(Nn=-1)), (1, dict(mb=0)), (1, dict(ps=0)), (1, dict(ps=96)), (1, dict(np=0)),
    (2, dict(B=65536)), (2, dict(mb=1 << 25)), (1, dict(bt=0)), (1, dict(sl=0)), (1, dict(fp=0)), (1, dict(fc=0)),
    (1, dict(no=0)), (1, dict(co=0)), (3, dict(bt=M + 2)), (3, dict(sl=2)), (3, dict(nl=2)), (3, dict(fp=2)),
    (3, dict(fc=2)), (3, dict(no=6 * M + 1)), (3, dict(so=2)), (3, dict(sm=8 * M + 4)), (3, dict(co=2)),
    (1, dict(co=5 * M)), (1, dict(so=2 * M + 12)), (1, dict(no=3 * M)), (1, dict(no=4 * M + 156)), (1, dict(sm=M)),
    (1, dict(no=7 * M)), (1, dict(bt=4 * M - 4)),
])
def test_reserve_argument_checks(L, want, kw):
    assert reserve(L, **kw) == want


def release(L, **kw):
    a = dict(bt=M, mb=8, ps=64, np=40, sl=2 * M, kl=3 * M, fp=4 * M, fc=5 * M, co=9 * M, B=4)
    a.update(kw)
    return L.attn_kvcache_release_paged(vp(a["bt"]), a["mb"], a["ps"], a["np"], vp(a["sl"]), vp(a["kl"]), vp(a["fp"]),
                                        vp(a["fc"]), vp(a["co"]), a["B"], None)


@pytest.mark.parametrize("want,kw", [
    (1, dict(B=0)), (1, dict(mb=0)), (1, dict(ps=65)), (1, dict(np=0)), (2, dict(B=1 << 17)), (1, dict(bt=0)),
    (1, dict(sl=0)), (1, dict(kl=0)), (1, dict(fp=0)), (1, dict(fc=0)), (1, dict(co=0)), (3, dict(kl=2)),
    (3, dict(co=9 * M + 2)), (1, dict(co=5 * M)), (1, dict(fp=M + 64)), (1, dict(co=4 * M + 8)),
])
def test_release_argument_checks(L, want, kw):
    assert release(L, **kw) == want


def bounds(L, **kw):
    a = dict(kp=1 << 32, kb=1 << 33, bt=M, mb=8, ps=128, np=40, sl=2 * M, nl=0, B=4, Nn=5, Hkv=2, d=64)
    a.update(kw)
    return L.attn_kvcache_bounds_paged(vp(a["kp"]), vp(a["kb"]), vp(a["bt"]), a["mb"], a["ps"], a["np"], vp(a["sl"]),
                                       vp(a["nl"]), a["B"], a["Nn"], a["Hkv"], a["d"], None)


@pytest.mark.parametrize("want,kw", [
    (0, dict(Nn=0)), (1, dict(Nn=-1)), (1, dict(B=0)), (1, dict(Hkv=0)), (2, dict(d=96)), (1, dict(ps=100)),
    (2, dict(Hkv=(1 << 20) + 1)), (1, dict(kp=0)), (1, dict(kb=0)), (1, dict(bt=0)), (1, dict(sl=0)), (3, dict(kp=24)),
    (3, dict(kb=40)), (3, dict(nl=2)), (2, dict(mb=1 << 25)), (1, dict(kb=(1 << 32) + 1024)),
])
def test_bounds_argument_checks(L, want, kw):
    assert bounds(L, **kw) == want


def select(L, **kw):
    a = dict(q=16, kb=16, bt=M, mb=8, ps=128, np=40, sl=2 * M, out=M, B=4, Nq=2, Hq=8, Hkv=2, d=64, topk=4, sink=1, local=1,
             ws=16, wsb=1 << 26)
    a.update(kw)
    return L.attn_select_blocks_paged(vp(a["q"]), vp(a["kb"]), vp(a["bt"]), a["mb"], a["ps"], a["np"], vp(a["sl"]),
                                      vp(a["out"]), a["B"], a["Nq"], a["Hq"], a["Hkv"], a["d"], a["topk"], a["sink"],
                                      a["local"], vp(a["ws"]), a["wsb"], None)


@pytest.mark.parametrize("want,kw", [
    (1, dict(B=0)), (1, dict(Nq=0)), (1, dict(Hq=7)), (1, dict(Hkv=0)), (2, dict(d=32)), (1, dict(ps=32)), (1, dict(topk=0)),
    (1, dict(sink=-1)), (1, dict(local=-1)), (1, dict(sink=3, local=2)), (1, dict(sink=(1 << 31) - 1, local=(1 << 31) - 1)),
    (2, dict(Hq=258)), (1, dict(q=0)), (1, dict(kb=0)), (1, dict(out=0)), (3, dict(q=8)), (3, dict(kb=8)), (3, dict(out=2)),
    (7, dict(ws=0)), (7, dict(ws=8)), (7, dict(wsb=64)), (2, dict(B=60000, Nq=60000)), (2, dict(mb=1 << 25)),
])
def test_selection_argument_checks(L, want, kw):
    assert select(L, **kw) == want


def attend(L, listed, **kw):
    a = dict(q=16, kp=16, vp=32, bt=M, mb=8, ps=128, np=40, sl=2 * M, x=M if listed else 256, n=4, o=1 << 30, lse=3 * M, B=4,
             Nq=2, Hq=8, Hkv=2, d=64, s=0.1, ws=16, wsb=1 << 30)
    a.update(kw)
    head = (vp(a["q"]), vp(a["kp"]), vp(a["vp"]), vp(a["bt"]), a["mb"], a["ps"], a["np"], vp(a["sl"]))
    tail = (vp(a["o"]), vp(a["lse"]), a["B"], a["Nq"], a["Hq"], a["Hkv"], a["d"], a["s"], vp(a["ws"]), a["wsb"], None)
    return (L.attn_fwd_blocks_paged(*head, vp(a["x"]), a["n"], *tail) if listed
            else L.attn_fwd_splitkv_paged_shared(*head, a["x"], *tail))


@pytest.mark.parametrize("listed", [False, True])
@pytest.mark.parametrize("want,kw", [
    (1, dict(B=0)), (1, dict(Nq=0)), (1, dict(Hq=9)), (1, dict(Hkv=0)), (2, dict(d=80)), (1, dict(mb=0)), (1, dict(np=0)),
    (1, dict(ps=96)), (1, dict(s=math.nan)), (1, dict(s=math.inf)), (2, dict(Hq=258)), (2, dict(B=65536)),
    (2, dict(B=60000, Nq=60000)), (2, dict(mb=1 << 25)), (2, dict(np=1 << 30)), (1, dict(q=0)), (1, dict(kp=0)),
    (1, dict(vp=0)), (1, dict(o=0)), (1, dict(lse=0)), (1, dict(bt=0)), (1, dict(sl=0)), (3, dict(q=24)), (3, dict(kp=24)),
    (3, dict(vp=24)), (3, dict(o=(1 << 30) + 8)), (3, dict(lse=2)), (3, dict(bt=2)), (3, dict(sl=2)), (1, dict(o=32)),
    (7, dict(ws=0)), (7, dict(ws=8)), (7, dict(wsb=1000)),
])
def test_attention_argument_checks(L, listed, want, kw):
    assert attend(L, listed, **kw) == want


@pytest.mark.parametrize("listed,want,kw", [
    (True, 1, dict(x=0)), (True, 3, dict(x=M + 2)), (True, 1, dict(n=0)), (True, 2, dict(n=513)),
    (False, 1, dict(x=-128)), (False, 1, dict(x=64)), (False, 1, dict(x=9 * 128)),
])
def test_list_and_prefix_checks(L, listed, want, kw):
    assert attend(L, listed, **kw) == want


def test_workspace_sizes(L):
    lists = lambda *a: L.attn_fwd_blocks_paged_workspace_size(*a, 4, 1024)
    for f in (L.attn_splitkv_paged_shared_workspace_size, lists):
        n = f(4, 2, 8, 2, 64)
        assert 0 < n < 1 << 28
        assert f(0, 2, 8, 2, 64) == f(4, 0, 8, 2, 64) == f(4, 2, 9, 2, 64) == f(4, 2, 8, 2, 65) == f(4, 2, 258, 2, 64) == 0
    assert attend(L, False, wsb=L.attn_splitkv_paged_shared_workspace_size(4, 2, 8, 2, 64) - 1) == 7
    assert attend(L, True, wsb=lists(4, 2, 8, 2, 64) - 1) == 7
    many = L.attn_fwd_blocks_paged_workspace_size(4, 600, 8, 2, 64, 16, 1024)  # sorted by block
    assert many > 600 * 8 * 16 * 65 * 4 and attend(L, True, Nq=600, n=16, o=1 << 40, wsb=many - 1) == 7
    n = L.attn_select_blocks_workspace_size(4, 2, 2, 1024)
    assert n >= 4 * 2 * 2 * 16 * 4 and select(L, wsb=n - 1) == 7
    assert L.attn_select_blocks_workspace_size(0, 2, 2, 1024) == L.attn_select_blocks_workspace_size(4, 2, 2, 63) == 0
    assert L.attn_fwd_blocks_paged_workspace_size(4, 2, 8, 2, 64, 0, 1024) == 0
    assert L.attn_fwd_blocks_paged_workspace_size(4, 2, 8, 2, 64, 513, 1024) == 0
    assert L.attn_fwd_blocks_paged_workspace_size(4, 2, 8, 2, 64, 4, 63) == 0
    # lists of few tokens, and those over many blocks, take the same whatever their number; others are sorted, with
    # what the entries give held for a chunk of the tokens
    wide = lambda Nq: L.attn_fwd_blocks_paged_workspace_size(1, Nq, 8, 2, 64, 32, 1 << 24)
    assert wide(4096) == wide(1)
    near = lambda Nq: L.attn_fwd_blocks_paged_workspace_size(1, Nq, 8, 2, 64, 32, 16384)
    assert near(16) == near(1) and near(4096) > 4096 * 8 * 32 * 65 * 4
    assert near(1 << 16) < (1 << 30) * 1.1 + (1 << 16) * 2 * 32 * 8


def test_the_binding_refuses_what_is_not_on_a_gpu_or_of_another_shape():
    q, kp = torch.zeros((1, 1, 2, 64), dtype=torch.bfloat16), torch.zeros((4, 64, 1, 64), dtype=torch.bfloat16)
    bt, sl = torch.zeros((1, 4), dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    for call in (lambda: A.decode_paged_shared(q, kp, kp, bt, sl, 0, 0.1),
                 lambda: A.attend_blocks_paged(q, kp, kp, bt, sl, torch.zeros((1, 1, 1, 2), dtype=torch.int32), 0.1),
                 lambda: A.select_blocks_paged(q, torch.zeros((4, 1, 1, 2, 64), dtype=torch.bfloat16), bt, sl, 2),
                 lambda: A.kvcache_bounds_paged(kp, kp, bt, sl, 1),
                 lambda: A.kvcache_reserve_paged(bt, sl, None, bt[0], sl, 64, 1),
                 lambda: A.kvcache_release_paged(bt, sl, sl, bt[0], sl, 64)):
        with pytest.raises(ValueError):
            call()


def test_definition_of_reserve_and_release():
    table, granted, slots, count = P.reserve([[5, -1, -1], [6, -1, -1], [7, -1, -1]], [10, 64, 64], [54, 2, 1], [1, 2, 3], 2,
                                             64, 54)
    assert table == [[5, -1, -1], [6, 2, -1], [7, 1, -1]] and granted == [54, 2, 1] and count == 0
    assert slots[0][:2] == [5 * 64 + 10, 5 * 64 + 11] and slots[1][:3] == [128, 129, -1] and slots[2][0] == 64
    free, count = P.release(table, [64, 66, 65], [10, 64, 64], [9, 9, 9], 0, 64)
    assert free == [1, 2, 9] and count == 2


def test_definition_of_bounds_bounds_every_key():
    g = torch.Generator().manual_seed(0)
    table, num = P.tables(g, 1, 3, 0)
    kp, = P.pools(g, num, 64, 1, 64, 1)
    kb = P.bounds(kp, table, 64, [150], [150], torch.zeros((num, 1, 1, 2, 64), dtype=torch.bfloat16))
    q = torch.randn((1, 1, 2, 64), generator=g).to(torch.bfloat16)
    flat = kb[table[0].long()].reshape(3, 2, 64)
    best = P.scores(q[0, 0], flat[:, 0], flat[:, 1])
    for j in range(3):
        keys = kp[table[0, j].long(), :min(64, 150 - 64 * j), 0].double()
        assert (q[0, 0].double() @ keys.T).max() <= best[j] + 1e-9


def test_definition_of_attention_against_a_softmax_over_all_keys():
    g = torch.Generator().manual_seed(1)
    table, num = P.tables(g, 1, 2, 0)
    kp, vp_ = P.pools(g, num, 64, 1, 64)
    q = torch.randn((1, 1, 2, 64), generator=g).to(torch.bfloat16)
    o, lse, _, _ = P.attend(q, kp, vp_, table, 64, 0.2, lambda b, i, h: list(range(100)))
    k, v = (x[table[0].long()].reshape(-1, 64)[:100].double() for x in (kp, vp_))
    s = 0.2 * q[0, 0].double() @ k.T
    assert torch.allclose(o[0, 0], torch.softmax(s, -1) @ v) and torch.allclose(lse[0, :, 0], torch.logsumexp(s, -1))

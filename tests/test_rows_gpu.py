"""Decode behind a shared prefix and attention over listed blocks, against 64 bits."""
import pytest
import torch

from tests import _paged as P
from exact_io_aware_14_gb300 import _native as A

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def make(seed, B, Nq, Hq, Hkv, d, page, shared, lens, stale=True):
    """q, pools and table on the CPU; NaN behind each sequence's end, in its last page and in the pages never used."""
    g = torch.Generator().manual_seed(seed)
    blocks = max(-(-max(lens) // page), shared // page, 1)
    table, num = P.tables(g, B, blocks, shared // page)
    kp, vp = P.pools(g, num, page, Hkv, d)
    if stale:
        used = torch.zeros((num, page), dtype=torch.bool)
        for b, L in enumerate(lens):
            n = torch.arange(L)
            used[table[b].long()[n // page], n % page] = True
        used[table[0, :shared // page].long()] = True
        kp[~used], vp[~used] = float("nan"), float("nan")
    return torch.randn((B, Nq, Hq, d), generator=g).to(torch.bfloat16), kp, vp, table


def seen(lens, Nq):
    return lambda b, i, h: list(range(max(0, lens[b] - Nq + 1 + i)))


def run_shared(q, kp, vp, table, lens, shared, scale, **kw):
    out = A.decode_paged_shared(q.cuda(), kp.cuda(), vp.cuda(), table.cuda(), i32(lens), shared, scale, **kw)
    assert A.attn_get_device_status() == 0
    return out


SHARED = [
    # B, Nq, Hq, Hkv, d, page, shared, lens
    (1, 1, 1, 1, 64, 64, 0, [1]),
    (1, 1, 1, 1, 128, 64, 64, [65]),
    (1, 1, 4, 1, 128, 64, 128, [128]),                         # nothing of its own
    (3, 1, 8, 2, 128, 64, 128, [129, 192, 193]),
    (3, 3, 9, 3, 64, 192, 192, [195, 392, 321]),
    (4, 2, 4, 2, 128, 64, 256, [257, 100, 0, 1]),              # shorter than the prefix, empty, one of two rows
    (2, 5, 2, 1, 64, 64, 0, [3, 200]),
    (40, 1, 8, 2, 128, 64, 320, [321 + 7 * (i % 9) for i in range(40)]),     # two tiles of rows
    (70, 1, 8, 2, 64, 64, 192, [193 + 40 * (i % 5) for i in range(70)]),     # three
    (3, 1, 7, 1, 128, 128, 128, [300, 129, 400]),
    (2, 1, 128, 1, 128, 64, 64, [150, 300]),                   # a group as large as a tile
    (2, 3, 100, 1, 64, 64, 64, [150, 300]),                    # one token a tile
    (2, 60, 6, 2, 128, 64, 128, [200, 331]),                   # more new rows than a tile
    (5, 1, 16, 16, 64, 64, 640, [641, 700, 1500, 642, 900]),
    (1, 1, 8, 2, 128, 64, 0, [5000]),
    (2, 1, 4, 1, 128, 256, 1536, [2500, 1537]),
    (700, 1, 2, 1, 64, 64, 64, [65 + i % 70 for i in range(700)]),   # more sequences than threads
    (400, 1, 40, 1, 64, 64, 0, [1 + i % 90 for i in range(400)]),    # the same, with more rows than few
]


@pytest.mark.parametrize("B,Nq,Hq,Hkv,d,page,shared,lens", SHARED)
def test_shared_prefix(B, Nq, Hq, Hkv, d, page, shared, lens):
    q, kp, vp, table = make(B + Nq + Hq, B, Nq, Hq, Hkv, d, page, shared, lens)
    scale = d ** -0.5
    o, lse = run_shared(q, kp, vp, table, lens, shared, scale)
    P.check(o, lse, P.attend(q, kp, vp, table, page, scale, seen(lens, Nq)))


@pytest.mark.parametrize("scale", [-0.3, 0.0, 3.0])
def test_scales(scale):
    lens = [300, 200, 129]
    q, kp, vp, table = make(1, 3, 2, 4, 2, 128, 64, 128, lens)
    want = P.attend(q, kp, vp, table, 64, scale, seen(lens, 2))
    P.check(*run_shared(q, kp, vp, table, lens, 128, scale), want)
    blocks = torch.tensor([[0, 1, 2, 3, 4]], dtype=torch.int32).expand(3, 2, 2, 5).contiguous()
    o, lse = A.attend_blocks_paged(*(x.cuda() for x in (q, kp, vp, table)), i32(lens), blocks.cuda(), scale)
    P.check(o, lse, want)


def test_scores_that_rise_along_the_keys():
    # the exponents' reference has to move again and again
    lens = [1500, 1100]
    q, kp, vp, table = make(2, 2, 1, 4, 1, 128, 64, 1024, lens, stale=False)
    q[:] = 1
    for b in range(2):
        n = torch.arange(lens[b])
        kp[table[b].long()[n // 64], n % 64, 0] = (n[:, None] / 16.0).to(torch.bfloat16)
    want = P.attend(q, kp, vp, table, 64, 0.5, seen(lens, 1))
    P.check(*run_shared(q, kp, vp, table, lens, 1024, 0.5), want)
    blocks = torch.arange(24, dtype=torch.int32).expand(2, 1, 1, 24).contiguous()
    o, lse = A.attend_blocks_paged(*(x.cuda() for x in (q, kp, vp, table)), i32(lens), blocks.cuda(), 0.5)
    P.check(o, lse, want)


def test_long_prefix_and_long_sequences():
    lens = [20000, 12289, 33000]
    q, kp, vp, table = make(3, 3, 1, 2, 1, 64, 256, 12288, lens)
    o, lse = run_shared(q, kp, vp, table, lens, 12288, 0.125)
    P.check(o, lse, P.attend(q, kp, vp, table, 256, 0.125, seen(lens, 1)))


def test_shared_results_repeat_bit_by_bit_and_whatever_the_memory_held():
    lens = [700, 650, 900]
    args = make(4, 3, 2, 8, 2, 128, 64, 640, lens)
    n = A.lib().attn_splitkv_paged_shared_workspace_size(3, 2, 8, 2, 128)
    outs = []
    for fill in (0, 255, 0x7f):
        ws = torch.full((n,), fill, dtype=torch.uint8, device="cuda")
        outs.append(run_shared(*args, lens, 640, 0.1, workspace=ws))
    for o, lse in outs[1:]:
        assert torch.equal(o, outs[0][0]) and torch.equal(lse, outs[0][1])


def guarded(n, dtype):
    """A tensor of n elements between 4096 bytes of a pattern, and what checks them."""
    size = n * torch.empty((), dtype=dtype).element_size()
    raw = torch.full((size + 8192,), 0x5A, dtype=torch.uint8, device="cuda")
    return raw[4096:4096 + size].view(dtype), lambda: bool((raw[:4096] == 0x5A).all() and (raw[4096 + size:] == 0x5A).all())


@pytest.mark.parametrize("kind", ["shared", "blocks"])
@pytest.mark.parametrize("B,Nq,Hq,Hkv,d", [(3, 1, 6, 2, 128), (2, 3, 5, 5, 64), (67, 1, 8, 2, 128), (1, 300, 7, 1, 64)])
def test_nothing_is_written_outside(kind, B, Nq, Hq, Hkv, d):
    lens = [400 + i % 7 for i in range(B)]
    q, kp, vp, table = (x.cuda() for x in make(5, B, Nq, Hq, Hkv, d, 64, 128, lens))
    shared, lists = A.lib().attn_splitkv_paged_shared_workspace_size, A.lib().attn_fwd_blocks_paged_workspace_size
    size = shared if kind == "shared" else lambda *a: lists(*a, 4, 64 * table.shape[1])
    ws, ok_ws = guarded(size(B, Nq, Hq, Hkv, d), torch.uint8)
    o, ok_o = guarded(q.numel(), torch.bfloat16)
    lse, ok_lse = guarded(B * Hq * Nq, torch.float32)
    sl = i32(lens)
    head = (q.data_ptr(), kp.data_ptr(), vp.data_ptr(), table.data_ptr(), table.shape[1], 64, kp.shape[0], sl.data_ptr())
    tail = (o.data_ptr(), lse.data_ptr(), B, Nq, Hq, Hkv, d, 0.1, ws.data_ptr(), ws.numel(),
            torch.cuda.current_stream().cuda_stream)
    if kind == "shared":
        assert A.lib().attn_fwd_splitkv_paged_shared(*head, 128, *tail) == 0
        want = P.attend(*(x.cpu() for x in (q, kp, vp, table)), 64, 0.1, seen(lens, Nq))
    else:
        blocks = torch.tensor([1, 3, 5, 6], dtype=torch.int32).expand(B, Nq, Hkv, 4).contiguous().cuda()
        assert A.lib().attn_fwd_blocks_paged(*head, blocks.data_ptr(), 4, *tail) == 0
        want = P.attend(*(x.cpu() for x in (q, kp, vp, table)), 64, 0.1,
                        lambda b, i, h: [k for j in (1, 3, 5, 6) for k in range(64 * j, min(64 * j + 64, lens[b] - Nq + 1 + i))])
    assert A.attn_get_device_status() == 0
    assert ok_ws() and ok_o() and ok_lse()
    P.check(o.view(B, Nq, Hq, d), lse.view(B, Hq, Nq), want)


def listed(blocks, lens, Nq):
    def keys(b, i, h):
        end = lens[b] - Nq + 1 + i
        return [k for j in blocks[b, i, h].tolist() if j >= 0 for k in range(64 * j, min(64 * j + 64, end))]
    return keys


def random_blocks(g, B, Nq, Hkv, n_sel, lens, full=True):
    out = torch.full((B, Nq, Hkv, n_sel), -1, dtype=torch.int32)
    for b in range(B):
        for i in range(Nq):
            nb = max(0, (lens[b] - Nq + i) // 64 + 1)
            for h in range(Hkv):
                pick = torch.randperm(nb, generator=g)[:n_sel].sort().values.to(torch.int32)
                if nb and not (pick == nb - 1).any():
                    pick[-1] = nb - 1
                out[b, i, h, :len(pick)] = pick
    return out


BLOCKS = [
    # B, Nq, Hq, Hkv, d, page, lens, n_sel
    (1, 1, 1, 1, 64, 64, [1], 1),
    (1, 1, 1, 1, 128, 64, [64], 3),
    (2, 1, 4, 2, 128, 64, [65, 1000], 4),
    (3, 3, 9, 3, 64, 192, [3, 700, 2000], 7),
    (2, 1, 128, 1, 128, 128, [900, 300], 5),
    (1, 1, 100, 1, 64, 64, [700], 6),
    (1, 1, 8, 8, 128, 256, [9000], 33),
    (2, 100, 4, 2, 128, 64, [150, 1111], 5),
    (1, 500, 6, 3, 64, 64, [500], 3),
    (1, 7, 16, 2, 128, 64, [5000], 70),
    (3, 2, 4, 2, 64, 64, [1, 0, 65], 2),
]


@pytest.mark.parametrize("B,Nq,Hq,Hkv,d,page,lens,n_sel", BLOCKS)
def test_listed_blocks(B, Nq, Hq, Hkv, d, page, lens, n_sel):
    q, kp, vp, table = make(B + Nq + n_sel, B, Nq, Hq, Hkv, d, page, 0, lens)
    blocks = random_blocks(torch.Generator().manual_seed(n_sel), B, Nq, Hkv, n_sel, lens)
    o, lse = A.attend_blocks_paged(*(x.cuda() for x in (q, kp, vp, table)), i32(lens), blocks.cuda(), d ** -0.5)
    assert A.attn_get_device_status() == 0
    P.check(o, lse, P.attend(q, kp, vp, table, page, d ** -0.5, listed(blocks, lens, Nq)))


# Many tokens on few blocks: sorted by block, and taken block by block.
BY_BLOCK = [
    (1, 900, 8, 2, 128, 64, [2100], 40),
    (2, 850, 6, 2, 64, 192, [850, 2900], 41),     # three heads: 126 rows a tile; lists that are not full
    (1, 1024, 8, 1, 128, 128, [1500], 64),
    (1, 700, 3, 3, 64, 64, [1000], 33),           # one head: tiles of 128 tokens
    (3, 1400, 5, 1, 128, 256, [5000, 100, 0], 47),  # tokens that see nothing, a sequence without keys
    (1, 600, 8, 1, 128, 64, [33100], 512),        # chunks of tokens
    (2, 256, 4, 1, 128, 64, [256, 700], 64),      # as few as are taken so
]


def by_block(Nq, Hq, Hkv, d, n_sel, keys):
    """Whether such a call is taken block by block: its workspace holds what each entry gives."""
    size = A.lib().attn_fwd_blocks_paged_workspace_size(1, Nq, Hq, Hkv, d, n_sel, keys)
    return size > 10 * A.lib().attn_fwd_blocks_paged_workspace_size(1, 1, Hq, Hkv, d, n_sel, keys)


@pytest.mark.parametrize("B,Nq,Hq,Hkv,d,page,lens,n_sel", BY_BLOCK)
def test_listed_blocks_of_many_tokens(B, Nq, Hq, Hkv, d, page, lens, n_sel):
    q, kp, vp, table = make(B + Nq + n_sel, B, Nq, Hq, Hkv, d, page, 0, lens)
    assert by_block(Nq, Hq, Hkv, d, n_sel, table.shape[1] * page)
    blocks = random_blocks(torch.Generator().manual_seed(n_sel), B, Nq, Hkv, n_sel, lens)
    o, lse = A.attend_blocks_paged(*(x.cuda() for x in (q, kp, vp, table)), i32(lens), blocks.cuda(), -0.1)
    assert A.attn_get_device_status() == 0
    P.check(o, lse, P.attend(q, kp, vp, table, page, -0.1, listed(blocks, lens, Nq)))


def prompt(seed=21, Nq=850, Hkv=2, n_sel=40, stale=True):
    lens = [1300]
    q, kp, vp, table = make(seed, 1, Nq, 4 * Hkv, Hkv, 128, 64, 0, lens, stale=stale)
    assert by_block(Nq, 4 * Hkv, Hkv, 128, n_sel, table.shape[1] * 64)
    g = torch.Generator().manual_seed(seed)
    # in any order, with blocks twice, behind the token and passed over
    blocks = torch.randint(-2, 1300 // 64 + 1, (1, Nq, Hkv, n_sel), generator=g, dtype=torch.int32)
    blocks[0, :200, :, 1:] = -1
    blocks[0, 100:120] = -1
    return lens, q, kp, vp, table, blocks


def test_lists_of_a_prompt_as_a_program_may_write_them():
    lens, q, kp, vp, table, blocks = prompt()
    for scale in (0.0, 0.1):
        o, lse = A.attend_blocks_paged(*(x.cuda() for x in (q, kp, vp, table)), i32(lens), blocks.cuda(), scale)
        assert A.attn_get_device_status() == 0
        P.check(o, lse, P.attend(q, kp, vp, table, 64, scale, listed(blocks, lens, 850)))


def test_values_that_are_not_numbers_behind_a_prompts_tokens():
    lens, q, kp, vp, table, blocks = prompt(22)
    blocks[0, 300:] = torch.where(blocks[0, 300:] == 2, 3, blocks[0, 300:])
    blocks[0, :300] = torch.where(blocks[0, :300] == 2, 1, blocks[0, :300])
    args = [x.cuda() for x in (q, kp, vp, table)]
    base = A.attend_blocks_paged(*args, i32(lens), blocks.cuda(), 0.1)
    P.check(*base, P.attend(q, kp, vp, table, 64, 0.1, listed(blocks, lens, 850)))

    def at(key):
        return args[3][0, key // 64].long(), key % 64
    args[1][at(130)[0]], args[2][at(130)[0]] = float("nan"), float("nan")  # a block that nobody lists
    args[1][at(1299)] = float("nan")
    args[2][at(1100)[0], at(1100)[1], 1, 77] = float("inf")
    args[2][at(1111)[0], at(1111)[1], 1, 77] = float("nan")
    args[2][at(1090)[0], at(1090)[1], 0, 5] = float("-inf")
    o, lse = A.attend_blocks_paged(*args, i32(lens), blocks.cuda(), 0.1)
    # what a token sees of them, and nothing else, is spoiled
    pos = torch.arange(850) + 1300 - 850
    lists = blocks[0].long()
    spoiled = torch.zeros((850, 8, 128), dtype=torch.bool)
    sees = lambda key, h: ((lists[:, h] == key // 64).any(-1) & (pos >= key))[:, None]
    spoiled[:, 4:, 77] = sees(1100, 1)
    spoiled[:, :4, 5] = sees(1090, 0)
    for h in range(2):
        spoiled[:, 4 * h:4 * h + 4] |= sees(1299, h)[..., None]
    spoiled = spoiled.cuda()
    assert spoiled.any(0).any(-1).all() and not spoiled.all(0).any()
    assert not o[0][spoiled].isfinite().any()
    assert torch.equal(o[0][~spoiled], base[0][0][~spoiled])
    assert torch.equal(lse[..., :849], base[1][..., :849])


def test_a_prompts_results_repeat_and_stay_inside_their_memory():
    lens, q, kp, vp, table, blocks = prompt(23)
    q, kp, vp, table, blocks = (x.cuda() for x in (q, kp, vp, table, blocks))
    size = A.lib().attn_fwd_blocks_paged_workspace_size(1, 850, 8, 2, 128, 40, 64 * table.shape[1])
    outs = []
    for fill in (0, 255, 0x7f):
        ws, ok_ws = guarded(size, torch.uint8)
        ws.fill_(fill)
        outs.append(A.attend_blocks_paged(q, kp, vp, table, i32(lens), blocks, 0.1, workspace=ws))
        assert A.attn_get_device_status() == 0 and ok_ws()
    for o, lse in outs[1:]:
        assert torch.equal(o, outs[0][0]) and torch.equal(lse, outs[0][1])


def test_a_captured_prompt_follows_its_inputs():
    lens, q, kp, vp, table, blocks = prompt(24, stale=False)
    args = [x.cuda() for x in (q, kp, vp, table)]
    sl, bl = i32(lens), blocks.cuda()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        A.attend_blocks_paged(*args, sl, bl, 0.1)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = A.attend_blocks_paged(*args, sl, bl, 0.1)
    for lens in ([1300], [600], [1299]):
        blocks = blocks.flip(1)
        sl.copy_(i32(lens))
        bl.copy_(blocks)
        graph.replay()
        torch.cuda.synchronize()
        P.check(o, lse, P.attend(q, kp, vp, table, 64, 0.1, listed(blocks, lens, 850)))
    assert A.attn_get_device_status() == 0


def test_bad_lengths_pages_and_blocks_of_a_prompt_are_reported():
    lens, q, kp, vp, table, blocks = prompt(25, stale=False)
    want = P.attend(q, kp, vp, table, 64, 0.1, listed(blocks, lens, 850))
    q, kp, vp, table, blocks = (x.cuda() for x in (q, kp, vp, table, blocks))
    for bad in (-1, 64 * table.shape[1] + 1):
        A.attend_blocks_paged(q, kp, vp, table, i32([bad]), blocks, 0.1)
        assert A.attn_get_device_status() == A.ATTN_ERR_DEVICE_ARG
    for bad in (-1, kp.shape[0]):
        other = table.clone()
        other[0, 3] = bad
        A.attend_blocks_paged(q, kp, vp, other, i32(lens), blocks, 0.1)
        assert A.attn_get_device_status() == A.ATTN_ERR_DEVICE_ARG
    for bad in (table.shape[1], 0x7fffffff):
        over = torch.where(blocks == -2, bad, blocks)
        o, lse = A.attend_blocks_paged(q, kp, vp, table, i32(lens), over, 0.1)
        assert A.attn_get_device_status() == A.ATTN_ERR_DEVICE_ARG
        P.check(o, lse, want)


@pytest.mark.parametrize("rows", [
    [[3, 1, 0, 2]],                       # any order
    [[-1, 2, -5, 0]],                     # passed over wherever they are
    [[-1, -1, -1, -1]],                   # nothing
    [[2, 2, 2, 0]],                       # the same block again counts again
    [[4, 5, 6, 7]],                       # behind the token's position
    [[7, 1, -1, 4]],
    [[3, 3, 3, 3]],
])
def test_lists_as_a_program_may_write_them(rows):
    lens = [230, 250]
    q, kp, vp, table = make(6, 2, 1, 4, 1, 128, 64, 512, lens, stale=False)
    table = torch.cat((table, table), 1)[:, :8].contiguous()
    blocks = torch.tensor(rows, dtype=torch.int32).expand(2, 1, 1, 4).contiguous()
    o, lse = A.attend_blocks_paged(*(x.cuda() for x in (q, kp, vp, table)), i32(lens), blocks.cuda(), 0.1)
    assert A.attn_get_device_status() == 0
    P.check(o, lse, P.attend(q, kp, vp, table, 64, 0.1, listed(blocks, lens, 1)))


def test_values_that_are_not_numbers_in_blocks_not_listed_or_behind_the_token():
    lens = [300]
    q, kp, vp, table = make(7, 1, 40, 4, 2, 128, 64, 0, lens)
    blocks = random_blocks(torch.Generator().manual_seed(1), 1, 40, 2, 3, lens)
    blocks = torch.where(blocks == 1, 0, blocks)
    want = P.attend(q, kp, vp, table, 64, 0.1, listed(blocks, lens, 40))
    first = (300 - 40) // 64 * 64  # rows differ in what they see of the last blocks
    base = A.attend_blocks_paged(*(x.cuda() for x in (q, kp, vp, table)), i32(lens), blocks.cuda(), 0.1)
    kp[table[0, 1].long()], vp[table[0, 1].long()] = float("nan"), float("inf")
    kp[table[0, 299 // 64].long(), 299 % 64], vp[table[0, 299 // 64].long(), 299 % 64] = float("inf"), float("nan")
    o, lse = A.attend_blocks_paged(*(x.cuda() for x in (q, kp, vp, table)), i32(lens), blocks.cuda(), 0.1)
    P.check(*base, want)
    assert first < 299
    # every token but the last, which alone sees the last key
    assert torch.equal(o[:, :39], base[0][:, :39]) and torch.equal(lse[..., :39], base[1][..., :39])
    assert bool(o[:, 39].isnan().any())


def test_bad_lengths_pages_and_blocks_are_reported():
    q, kp, vp, table = (x.cuda() for x in make(8, 2, 1, 4, 2, 64, 64, 64, [200, 130], stale=False))
    blocks = i32([[[[0, 1]] * 2]] * 2)
    for lens in ([-1, 100], [100, 257]):
        A.decode_paged_shared(q, kp, vp, table, i32(lens), 64, 0.1)
        assert A.attn_get_device_status() == A.ATTN_ERR_DEVICE_ARG
        A.attend_blocks_paged(q, kp, vp, table, i32(lens), blocks, 0.1)
        assert A.attn_get_device_status() == A.ATTN_ERR_DEVICE_ARG
    bad = table.clone()
    bad[1, 1] = kp.shape[0]
    A.decode_paged_shared(q, kp, vp, bad, i32([200, 130]), 64, 0.1)
    assert A.attn_get_device_status() == A.ATTN_ERR_DEVICE_ARG
    A.attend_blocks_paged(q, kp, vp, bad, i32([200, 130]), blocks, 0.1)
    assert A.attn_get_device_status() == A.ATTN_ERR_DEVICE_ARG
    o, lse = A.attend_blocks_paged(q, kp, vp, table, i32([200, 130]), i32([[[[0, 9]] * 2]] * 2), 0.1)
    assert A.attn_get_device_status() == A.ATTN_ERR_DEVICE_ARG
    one = A.attend_blocks_paged(q, kp, vp, table, i32([200, 130]), i32([[[[0]] * 2]] * 2), 0.1)
    P.check(o, lse, P.attend(*(x.cpu() for x in (q, kp, vp, table)), 64, 0.1, lambda b, i, h: list(range(64))))
    P.check(*one, P.attend(*(x.cpu() for x in (q, kp, vp, table)), 64, 0.1, lambda b, i, h: list(range(64))))


def test_captured_calls_follow_their_inputs():
    lens0, lens1 = [300, 140, 520], [129, 513, 256]
    q, kp, vp, table = (x.cuda() for x in make(9, 3, 1, 8, 2, 128, 64, 128, [520] * 3, stale=False))
    sl = i32(lens0)
    blocks = random_blocks(torch.Generator().manual_seed(3), 3, 1, 2, 3, [129] * 3).cuda()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        A.decode_paged_shared(q, kp, vp, table, sl, 128, 0.1)
        A.attend_blocks_paged(q, kp, vp, table, sl, blocks, 0.1)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a = A.decode_paged_shared(q, kp, vp, table, sl, 128, 0.1)
        c = A.attend_blocks_paged(q, kp, vp, table, sl, blocks, 0.1)
    host = [x.cpu() for x in (q, kp, vp, table)]
    for lens in (lens1, lens0, lens1):
        sl.copy_(i32(lens))
        graph.replay()
        torch.cuda.synchronize()
        P.check(*a, P.attend(*host, 64, 0.1, seen(lens, 1)))
        P.check(*c, P.attend(*host, 64, 0.1, listed(blocks.cpu(), lens, 1)))
    assert A.attn_get_device_status() == 0


def test_calls_at_once_on_two_streams():
    lens = [900, 700]
    args = [[x.cuda() for x in make(10 + i, 2, 1, 8, 2, 128, 64, 640, lens)] for i in range(2)]
    want = [P.attend(*(x.cpu() for x in a), 64, 0.1, seen(lens, 1)) for a in args]
    sl, streams = i32(lens), [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            outs[i].append(A.decode_paged_shared(*args[i], sl, 640, 0.1, stream=s))
    torch.cuda.synchronize()
    assert A.attn_get_device_status() == 0
    for i in range(2):
        for o, lse in outs[i]:
            P.check(o, lse, want[i])


def test_a_serving_step_selects_what_it_attends_to():
    """Pages, keys, bounds, selection, attention: with room for every block the result is the dense one."""
    g = torch.Generator().manual_seed(11)
    B, Hq, Hkv, d, page, num = 3, 8, 2, 128, 64, 64
    kp, vp = (torch.zeros((num, page, Hkv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    kb = torch.zeros((num, 1, Hkv, 2, d), dtype=torch.bfloat16, device="cuda")
    table = torch.full((B, 16), -1, dtype=torch.int32, device="cuda")
    free, count = torch.randperm(num, generator=g).to(torch.int32).cuda(), i32([num])
    lens, keys, vals = i32([0] * B), [[] for _ in range(B)], [[] for _ in range(B)]
    for new in ([300, 64, 129], [1, 1, 1], [1, 1, 1], [3, 0, 2]):
        n = max(new)
        k, v, q = (torch.randn((B, n, h, d), generator=g).to(torch.bfloat16) for h in (Hkv, Hkv, Hq))
        granted, slots, count = A.kvcache_reserve_paged(table, lens, i32(new), free, count, page, n)
        after = torch.empty_like(lens)
        A.kvcache_append_paged(k.cuda(), v.cuda(), kp, vp, table, lens, new_lens=granted, seqlens_out=after)
        A.kvcache_bounds_paged(kp, kb, table, after, n, new_lens=granted)
        lens = after
        for b in range(B):
            keys[b].append(k[b, :new[b]])
            vals[b].append(v[b, :new[b]])
        at = slots[0, 0].item()
        assert torch.equal(kp.view(-1, Hkv, d)[at].cpu(), k[0, 0])
        q1 = q[:, :1].contiguous().cuda()
        dense = A.decode_paged_shared(q1, kp, vp, table, lens, 0, 0.1)
        all_ = A.attend_blocks_paged(q1, kp, vp, table, lens, A.select_blocks_paged(q1, kb, table, lens, 16), 0.1)
        few = A.select_blocks_paged(q1, kb, table, lens, 3)
        some = A.attend_blocks_paged(q1, kp, vp, table, lens, few, 0.1)
        assert A.attn_get_device_status() == 0
        host = [x.cpu() for x in (q1, kp, vp, table)]
        want = P.attend(*host, page, 0.1, seen(lens.tolist(), 1))
        P.check(*dense, want)
        P.check(*all_, want)
        assert torch.equal(few.cpu(), P.select(host[0], kb.cpu(), host[3], page, lens.tolist(), 3, 1, 1))
        P.check(*some, P.attend(*host, page, 0.1, listed(few.cpu(), lens.tolist(), 1)))
    c = A.kvcache_release_paged(table, lens, i32([0] * B), free, count, page)
    assert int(c) == num and sorted(free.tolist()) == list(range(num))


def test_a_prompt_selects_what_it_attends_to():
    """The same for the chunks of a prompt, the second behind the first's keys; then the rejected part is given back."""
    g = torch.Generator().manual_seed(12)
    Hq, Hkv, d, page, num = 8, 2, 64, 64, 24
    kp, vp = (torch.zeros((num, page, Hkv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    kb = torch.zeros((num, 1, Hkv, 2, d), dtype=torch.bfloat16, device="cuda")
    table = torch.full((1, 20), -1, dtype=torch.int32, device="cuda")
    free, count = torch.randperm(num, generator=g).to(torch.int32).cuda(), i32([num])
    lens, n = i32([0]), 600
    assert by_block(n, Hq, Hkv, d, 16, 20 * page)
    for chunk in range(2):
        k, v, q = (torch.randn((1, n, h, d), generator=g).to(torch.bfloat16).cuda() for h in (Hkv, Hkv, Hq))
        granted, _, count = A.kvcache_reserve_paged(table, lens, i32([n]), free, count, page, n)
        after = torch.empty_like(lens)
        A.kvcache_append_paged(k, v, kp, vp, table, lens, new_lens=granted, seqlens_out=after)
        A.kvcache_bounds_paged(kp, kb, table, after, n, new_lens=granted)
        lens = after
        blocks = A.select_blocks_paged(q, kb, table, lens, 16, 1, 2)
        o, lse = A.attend_blocks_paged(q, kp, vp, table, lens, blocks, 0.125)
        assert A.attn_get_device_status() == 0
        host = [x.cpu() for x in (q, kp, vp, table)]
        assert torch.equal(blocks.cpu(), P.select(host[0], kb.cpu(), host[3], page, lens.tolist(), 16, 1, 2))
        P.check(o, lse, P.attend(*host, page, 0.125, listed(blocks.cpu(), lens.tolist(), n)))
    count = A.kvcache_release_paged(table, lens, i32([n]), free, count, page)
    assert int(count) == num - 10 and A.attn_get_device_status() == 0

"""GPU: split-KV decode over a paged e4m3 cache against attention in 64 bits
over the values that the codes and scales stand for."""
import pytest
import torch

from exact_io_aware_14_gb300 import _native, build as native_build
from tests import _serving as S

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    native_build.build()
    _native.lib()
    torch.cuda.init()


def _cache(B, Hkv, d, page, lens, seed, amp=1.0, pow2=True, spread=3, extra=2, cap=None):
    """Pools, scales, table on the CPU; codes behind a sequence's end and of free pages are NaN."""
    g = torch.Generator().manual_seed(seed)
    mb = max(1, -(-(cap or max(lens)) // page))
    num_pages = B * mb + extra
    table = torch.randperm(num_pages, generator=g)[:B * mb].view(B, mb).to(torch.int32)
    pools, scales = [], []
    for _ in range(2):
        x = torch.randn((num_pages, page, Hkv, d), generator=g)
        s = amp * torch.exp2(torch.randint(-spread, spread + 1, (num_pages, Hkv), generator=g).float() - 6)
        if not pow2:
            s = s * (1 + torch.rand((num_pages, Hkv), generator=g))
        codes = (x * amp / s[:, None, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        live = torch.zeros((num_pages, page), dtype=torch.bool)
        for b in range(B):
            for blk in range(mb):
                live[table[b, blk], :max(0, min(page, lens[b] - blk * page))] = True
        codes[~live] = 0x7F
        pools.append(codes)
        scales.append(s)
    return g, pools, scales, table


def _run(q, pools, scales, table, lens, scale, chunk=None, **kw):
    return _native.decode_paged_fp8(q.cuda(), *(p.cuda().view(torch.float8_e4m3fn) for p in pools),
                                    *(s.cuda() for s in scales), table.cuda(),
                                    torch.tensor(lens, dtype=torch.int32).cuda(), scale, chunk, **kw)


def _check(q, pools, scales, table, lens, scale, got, what):
    n = max(max(lens), 1)
    k, v = (S.paged_rows(p.view(torch.float8_e4m3fn).double() * s.double()[:, None, :, None], table, n)
            for p, s in zip(pools, scales))
    o, lse, eo, el = S.decode(q, k, v, lens, scale)
    S.assert_within(got[0], o, eo + 2.0 ** -8 * (o.abs() + eo), what + " o")
    empty = lse.isinf()
    L = got[1].double().cpu()
    assert torch.equal(L == -float("inf"), empty), what
    S.assert_within(torch.where(empty, torch.zeros_like(L), L), torch.where(empty, torch.zeros_like(lse), lse), el,
                    what + " lse")


CASES = [
    # B, Nq, Hq, Hkv, d, page, lens, chunk
    (1, 1, 1, 1, 64, 64, [1], 64),
    (3, 1, 4, 1, 128, 64, [1, 64, 65], 128),
    (2, 1, 32, 8, 128, 256, [700, 1025], None),
    (4, 1, 8, 8, 128, 64, [127, 128, 129, 300], 256),
    (3, 1, 6, 2, 64, 192, [191, 192, 500], 128),
    (2, 1, 16, 1, 128, 128, [333, 1], 192),
    (2, 1, 40, 1, 64, 64, [210, 64], 64),
    (2, 1, 5, 1, 128, 320, [640, 77], 448),
    (3, 2, 8, 2, 128, 64, [1, 2, 200], 64),
    (2, 3, 24, 4, 64, 192, [3, 700], 256),
    (3, 4, 7, 7, 128, 64, [4, 131, 66], 64),
    (2, 7, 16, 2, 64, 128, [513, 7], 128),
    (1, 64, 2, 1, 64, 64, [130], 64),
    (2, 1, 18, 1, 128, 64, [300, 65], 128),          # 18 rows: three groups, the last with two
    (2, 3, 18, 3, 64, 192, [3, 500], 256),
    (2, 7, 24, 3, 128, 64, [7, 400], 192),           # 56 rows: blocks of 24, the last with one real group
    (1, 7, 16, 1, 64, 64, [200], 64),
    (4, 5, 4, 2, 128, 64, [0, 1, 3, 68], 64),       # rows that see no key, a sequence without any
]


@pytest.mark.parametrize("B,Nq,Hq,Hkv,d,page,lens,chunk", CASES)
def test_decode(B, Nq, Hq, Hkv, d, page, lens, chunk):
    g, pools, scales, table = _cache(B, Hkv, d, page, lens, 500 + Hq + d + page)
    q = torch.randn((B, Nq, Hq, d), generator=g).to(torch.bfloat16)
    got = _run(q, pools, scales, table, lens, d ** -0.5, chunk)
    assert _native.attn_get_device_status() == 0
    _check(q, pools, scales, table, lens, d ** -0.5, got, "decode")


@pytest.mark.parametrize("scale", [-0.11, 0.0, 1.0])
def test_scales_of_any_size(scale):
    """Scales that are no powers of two and differ by 2^12 between pages; a negative, zero and large softmax scale."""
    lens = [900, 257]
    g, pools, scales, table = _cache(2, 2, 128, 64, lens, 71, pow2=False, spread=6)
    q = torch.randn((2, 1, 8, 128), generator=g).to(torch.bfloat16)
    got = _run(q, pools, scales, table, lens, scale, 256)
    _check(q, pools, scales, table, lens, scale, got, "scales")


@pytest.mark.parametrize("size", [2.0 ** -120, 1e-41, 2.0 ** 60])
def test_value_scales_at_the_ends_of_the_range(size):
    """Value scales near the smallest normal number, below it, and large: o follows them."""
    lens = [200]
    g, pools, scales, table = _cache(1, 1, 128, 64, lens, 82)
    q = torch.randn((1, 1, 4, 128), generator=g).to(torch.bfloat16)
    scales[1] = torch.full_like(scales[1], size)
    scales[1][table[0, 1]] *= 0.5
    n = max(lens)
    k, v = (S.paged_rows(p.view(torch.float8_e4m3fn).double() * s.double()[:, None, :, None], table, n)
            for p, s in zip(pools, scales))
    o, lse, eo, el = S.decode(q, k, v, lens, 0.09)
    got = _run(q, pools, scales, table, lens, 0.09, 128)
    # fp32 on the way: multiples of 2^-149 at the least, and bf16 below 2^-126 has steps of 2^-133
    S.assert_within(got[0], o, eo + 2.0 ** -8 * (o.abs() + eo) + (2.0 ** -133 if size < 1 else 0), "o")
    S.assert_within(got[1], lse, el, "lse")


@pytest.mark.parametrize("Hq,Hkv,Nq,d", [(4, 1, 1, 128), (8, 1, 1, 64), (12, 1, 1, 128), (8, 1, 3, 64)])
@pytest.mark.parametrize("apart", [20, 27, 40, 60, 95])
def test_value_scales_far_apart(Hq, Hkv, Nq, d, apart):
    """Value scales 2^20 to 2^95 apart within a split, the softmax on the page with the smallest: its values are the
    result as long as the others' weights leave them so, wherever the page lies."""
    page, n, scale = 64, 400, d ** -0.5
    for at in (0, 1, 2, 6):
        g, pools, scales, table = _cache(1, Hkv, d, page, [n], 600 + at)
        q = torch.randn((1, Nq, Hq, d), generator=g).abs().to(torch.bfloat16)
        scales[0].fill_(2.0 ** -6)
        pools[0][table[0, at], :min(page, n - at * page)] = 0x7E   # 448: scores higher by 40 or more
        scales[1].fill_(1.0)
        scales[1][table[0, at]] = 2.0 ** -apart
        for chunk in (64, 128, 512):
            o, lse = _run(q, pools, scales, table, [n], scale, chunk)
            k, v = (S.paged_rows(p.view(torch.float8_e4m3fn).double() * s.double()[:, None, :, None], table, n)
                    for p, s in zip(pools, scales))
            vs = scales[1].double()[table[0].long()].repeat_interleave(page, 0)[:n, 0]
            for i in range(Nq):
                m = n - Nq + 1 + i
                kk, vv = k[0, :m, 0], v[0, :m, 0]
                for h in range(Hq):
                    qq = q[0, i, h].double()
                    s = scale * (kk @ qq)
                    p = torch.softmax(s, 0)
                    ds = 2.0 ** -23 * d * scale * float((kk.abs() @ qq.abs()).max())
                    top = float((p * vs[:m]).max())   # the largest weight with its scale
                    want = p @ vv
                    # weights: 9 bits, moved by the scores' error; what e5m2 drops: 2^-26 of the largest weight for
                    # each code; 2^-20 of the largest product for fp32 sums
                    err = (2.0 ** -9 + 2 * ds) * (p @ vv.abs()) + 2.0 ** -26 * top * (vv.abs() / vs[:m, None]).sum(0) \
                        + 2.0 ** -20 * top * 448
                    S.assert_within(o[0, i, h], want, err + 2.0 ** -8 * (want.abs() + err),
                                    "o, page %d, chunk %d, row %d, head %d" % (at, chunk, i, h))
                    L = float(torch.logsumexp(s, 0))
                    assert abs(float(lse[0, h, i]) - L) <= ds + 2.0 ** -20 * (1 + abs(L) + apart)


def test_zero_scales():
    """Pages whose scale is zero hold zeros: their keys score 0 and add nothing to o."""
    lens = [300]
    g, pools, scales, table = _cache(1, 2, 64, 64, lens, 72)
    scales[0][table[0, 1]] = 0.0
    scales[1][table[0, 2]] = 0.0
    q = torch.randn((1, 1, 4, 64), generator=g).to(torch.bfloat16)
    _check(q, pools, scales, table, lens, 0.125, _run(q, pools, scales, table, lens, 0.125, 128), "zero scales")
    for s in scales:
        s.zero_()
    _check(q, pools, scales, table, lens, 0.125, _run(q, pools, scales, table, lens, 0.125, 128), "all zero")


@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_rising_scores(sign):
    """Scores that climb by about 60 along the sequence: the softmax's reference moves many times in a split."""
    B, Hq, Hkv, d, page, lens = 2, 8, 2, 128, 64, [1500, 700]
    g, pools, scales, table = _cache(B, Hkv, d, page, lens, 73)
    q = torch.ones((B, 1, Hq, d), dtype=torch.bfloat16)
    scales[0].fill_(2.0 ** -6)
    for b in range(B):
        ramp = torch.linspace(-4, 4, lens[b]) * 64
        for blk in range(-(-lens[b] // page)):
            r = ramp[blk * page:(blk + 1) * page]
            pools[0][table[b, blk], :len(r)] = r[:, None, None].expand(-1, Hkv, d).to(torch.float8_e4m3fn).view(
                torch.uint8)
    got = _run(q, pools, scales, table, lens, sign * d ** -0.5, 1024)
    _check(q, pools, scales, table, lens, sign * d ** -0.5, got, "rising")


def test_peaked_and_wide_queries():
    """Queries whose values differ by 2^20 within a row, and rows where one key outweighs all others."""
    lens = [400, 130]
    g, pools, scales, table = _cache(2, 1, 64, 64, lens, 74)
    q = torch.randn((2, 1, 4, 64), generator=g)
    q = q * torch.exp2(-torch.randint(0, 21, q.shape, generator=g).float())
    q[1] *= 100
    q[0, 0, 3] = 0
    q = q.to(torch.bfloat16)
    _check(q, pools, scales, table, lens, 0.125, _run(q, pools, scales, table, lens, 0.125, 128), "wide")


def test_splits_and_repeats():
    """Results do not depend on a sequence's neighbours, and the same call gives the same bits; every split length
    stays inside the bounds."""
    lens = [1000, 1, 321]
    g, pools, scales, table = _cache(3, 2, 128, 64, lens, 75)
    q = torch.randn((3, 2, 8, 128), generator=g).to(torch.bfloat16)
    for chunk in (64, 192, 512, 2048):
        a = _run(q, pools, scales, table, lens, 0.09, chunk)
        b = _run(q, pools, scales, table, lens, 0.09, chunk)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        _check(q, pools, scales, table, lens, 0.09, a, "chunk %d" % chunk)
        c = _run(q[2:], pools, scales, table[2:], lens[2:], 0.09, chunk)
        assert torch.equal(a[0][2:], c[0]) and torch.equal(a[1][2:], c[1])
    assert _native.attn_get_device_status() == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [449, 600, 1500, 2048, 2113, 4200])
def test_long_rows_do_not_depend_on_batch_or_table(d, n):
    """A row of 8 to 66 splits: the same bits alone, among many rows and behind a wider table, and within its bounds."""
    Hq, Hkv, chunk = 4, 2, 64
    g, pools, scales, table = _cache(1, Hkv, d, 64, [n], 610 + n)
    q = torch.randn((1, 1, Hq, d), generator=g).to(torch.bfloat16)
    alone = _run(q, pools, scales, table, [n], 0.1, chunk)
    _check(q, pools, scales, table, [n], 0.1, alone, "alone")
    for cap in (n, 2112, 5000):
        t = torch.zeros((1, max(table.shape[1], -(-cap // 64))), dtype=torch.int32)
        t[:, :table.shape[1]] = table
        wide = _run(q, pools, scales, t, [n], 0.1, chunk)
        many = _run(q.repeat(160, 1, 1, 1), pools, scales, t.repeat(160, 1), [n] * 160, 0.1, chunk)
        for a, b, c in zip(alone, wide, many):
            assert torch.equal(a, b) and torch.equal(a.expand(160, *a.shape[1:]), c), "table of %d keys" % cap
    assert _native.attn_get_device_status() == 0


LONG = [
    # B, Nq, Hq, Hkv, d, page, lens, chunk
    (4, 1, 8, 2, 128, 64, [2200, 0, 40, 100], 64),      # 35 splits, few rows; neighbours of no, one and two splits
    (4, 1, 8, 2, 64, 64, [4200, 0, 64, 65], 64),        # 66
    (80, 1, 4, 2, 128, 64, [2200, 0, 40, 100] + [70] * 76, 64),   # more rows than twice the SMs: whole rows
    (80, 1, 4, 2, 64, 128, [4200, 0, 64, 65] + [130] * 76, 64),
    (2, 1, 2, 1, 128, 256, [17001, 16384], 64),         # 266 and 256 splits
    (2, 3, 2, 2, 64, 64, [16500, 2], 64),               # 258; new tokens that see nothing beside it
    (2, 1, 8, 2, 128, 64, [2100, 2048], 2048),          # a split of 32 pages
    (1, 1, 24, 1, 64, 64, [4097], 2048),
    (1, 1, 4, 1, 128, 256, [70001], None),              # far into a sequence
    (1, 2, 3, 1, 64, 64, [66000], 1024),
]


@pytest.mark.parametrize("B,Nq,Hq,Hkv,d,page,lens,chunk", LONG)
def test_long_sequences(B, Nq, Hq, Hkv, d, page, lens, chunk):
    """Many splits (each form of the combine, its second round of splits), splits of 2048 keys, long sequences."""
    g, pools, scales, table = _cache(B, Hkv, d, page, lens, 620 + d + page)
    q = torch.randn((B, Nq, Hq, d), generator=g).to(torch.bfloat16)
    got = _run(q, pools, scales, table, lens, d ** -0.5, chunk)
    assert _native.attn_get_device_status() == 0
    few = B if B <= 4 else 4      # the neighbours behind the fourth are there for their number
    _check(q[:few], pools, scales, table[:few], lens[:few], d ** -0.5, [x[:few] for x in got], "long")


@pytest.mark.parametrize("Hq,Hkv,Nq,d", [(4, 1, 1, 128), (8, 1, 1, 64), (16, 1, 1, 128), (18, 1, 1, 64), (6, 2, 2, 64)])
@pytest.mark.parametrize("cap,chunk", [(128, 64), (192, 64), (320, 64), (512, 64), (640, 128)])
def test_clusters_of_splits(Hq, Hkv, Nq, d, cap, chunk):
    """Two to eight splits that one cluster takes (ranks beyond the splits, splits behind a sequence's end, sequences
    without a key), against 64 bits and, bit for bit, the same splits among so many sequences that the combine
    kernel merges them."""
    lens = [cap, 1, 0, cap - 65, 64]
    g, pools, scales, table = _cache(5, Hkv, d, 64, lens, 83 + cap, cap=cap)
    q = torch.randn((5, Nq, Hq, d), generator=g).to(torch.bfloat16)
    got = _run(q, pools, scales, table, lens, 0.1, chunk)
    assert _native.attn_get_device_status() == 0
    _check(q, pools, scales, table, lens, 0.1, got, "clusters")
    many = 64
    big = _run(q.repeat(many, 1, 1, 1), pools, scales, table.repeat(many, 1), lens * many, 0.1, chunk)
    for a, b in zip(big, got):
        assert torch.equal(a.view(many, 5, *a.shape[1:]), b.expand(many, *b.shape))
    assert _native.attn_get_device_status() == 0


@pytest.mark.parametrize("B", [33, 70, 300])
def test_many_sequences(B):
    g0 = torch.Generator().manual_seed(B)
    lens = torch.randint(0, 200, (B,), generator=g0).tolist()
    lens[0], lens[-1] = 193, 0
    g, pools, scales, table = _cache(B, 1, 64, 64, lens, 76, cap=256)
    q = torch.randn((B, 1, 3, 64), generator=g).to(torch.bfloat16)
    _check(q, pools, scales, table, lens, 0.125, _run(q, pools, scales, table, lens, 0.125, 64), "B%d" % B)


def test_nan_in_the_cache_spoils_its_sequence_only():
    lens = [300, 200]
    g, pools, scales, table = _cache(2, 1, 128, 64, lens, 77)
    q = torch.randn((2, 1, 4, 128), generator=g).to(torch.bfloat16)
    pools[1][table[0, 1], 5, 0, 17] = 0x7F     # a value of sequence 0
    o, lse = _run(q, pools, scales, table, lens, 0.09, 128)
    assert o[0, :, :, 17].isnan().all() and o[0, :, :, :17].isfinite().all() and o[1].isfinite().all()
    assert lse.isfinite().all()
    pools[0][table[1, 0], 3, 0, 0] = 0x7F      # a key of sequence 1
    o, lse = _run(q, pools, scales, table, lens, 0.09, 128)
    assert o[1].isnan().all() and lse[1].isnan().all() and lse[0].isfinite().all()


def test_queries_that_are_not_finite():
    """A NaN or an infinity in a query row spoils that row only."""
    lens = [300]
    g, pools, scales, table = _cache(1, 2, 64, 64, lens, 84)
    q = torch.randn((1, 2, 8, 64), generator=g).to(torch.bfloat16)
    want = _run(q, pools, scales, table, lens, 0.125, 128)
    bad = q.clone()
    bad[0, 0, 1, 7] = float("nan")
    bad[0, 1, 6, 60] = float("-inf")
    o, lse = _run(bad, pools, scales, table, lens, 0.125, 128)
    spoilt = torch.zeros((2, 8), dtype=torch.bool)
    spoilt[0, 1] = spoilt[1, 6] = True
    assert o[0][spoilt].isnan().all() and lse[0].t()[spoilt].isnan().all()
    assert torch.equal(o[0][~spoilt], want[0][0][~spoilt]) and torch.equal(lse[0].t()[~spoilt], want[1][0].t()[~spoilt])


@pytest.mark.parametrize("Hq,Hkv", [(2, 1), (8, 1), (24, 1)])
def test_nan_among_the_new_tokens(Hq, Hkv):
    """A NaN in a value that only the last of the new tokens sees leaves the others as they are."""
    lens, Nq, d = [131], 3, 128
    g, pools, scales, table = _cache(1, Hkv, d, 64, lens, 79)
    q = torch.randn((1, Nq, Hq, d), generator=g).to(torch.bfloat16)
    want = _run(q, pools, scales, table, lens, 0.09, 128)
    spoilt = [p.clone() for p in pools]
    spoilt[1][table[0, 2], 2, 0, 17] = 0xFF    # the value of key 130
    o, lse = _run(q, spoilt, scales, table, lens, 0.09, 128)
    assert torch.equal(o[:, :2], want[0][:, :2]) and torch.equal(lse, want[1])
    assert o[:, 2].isnan().any(-1).all()
    spoilt = [p.clone() for p in pools]
    spoilt[0][table[0, 2], 2, 0, 5] = 0x7F     # its key
    o, lse = _run(q, spoilt, scales, table, lens, 0.09, 128)
    assert torch.equal(o[:, :2], want[0][:, :2]) and torch.equal(lse[..., :2], want[1][..., :2])
    assert o[:, 2].isnan().all() and lse[..., 2].isnan().all()


@pytest.mark.parametrize("Hq,Hkv,d", [(2, 1, 128), (8, 1, 64), (24, 1, 128), (6, 3, 64)])
@pytest.mark.parametrize("n,chunk", [(131, 128), (129, 128), (129, 64), (300, 512), (258, 128), (66, 64)])
def test_nan_values_among_the_new_tokens_stay_in_their_dimension(Hq, Hkv, d, n, chunk):
    """A NaN in a value that only some of the new tokens see: NaN in that dimension for those that see it, every other
    value as if it were a number."""
    Nq = 3
    g, pools, scales, table = _cache(2, Hkv, d, 64, [n, 40], 85)
    q = torch.randn((2, Nq, Hq, d), generator=g).to(torch.bfloat16)
    G = Hq // Hkv
    spots = [(n - 1, 17, 0), (n - 1, 63, Hkv - 1), (n - 2, 5, 0), (n - 2, 17, 0), (n - 4, 44, Hkv - 1)]
    clean, bad = [p.clone() for p in pools], [p.clone() for p in pools]
    hit = torch.zeros((2, Nq, Hq, d), dtype=torch.bool)
    for j, c, h in spots:
        clean[1][table[0, j // 64], j % 64, h, c] = 0
        bad[1][table[0, j // 64], j % 64, h, c] = 0xFF if c == 17 else 0x7F
        hit[0, max(0, j - (n - Nq)):, h * G:(h + 1) * G, c] = True
    want = _run(q, clean, scales, table, [n, 40], 0.09, chunk)
    o, lse = _run(q, bad, scales, table, [n, 40], 0.09, chunk)
    o, w = o.cpu(), want[0].cpu()
    assert o[hit].isnan().all()
    assert torch.equal(o[~hit], w[~hit]) and torch.equal(lse, want[1])
    assert _native.attn_get_device_status() == 0


def test_bad_lengths_and_pages_are_reported():
    lens = [300, 200]
    g, pools, scales, table = _cache(2, 1, 128, 64, lens, 78)
    q = torch.randn((2, 1, 4, 128), generator=g).to(torch.bfloat16)
    for bad in (-1, table.max().item() + 1000, 2 ** 31 - 1):
        t = table.clone()
        t[0, 1] = bad
        o, _ = _run(q, pools, scales, t, lens, 0.09, 128)
        assert _native.attn_get_device_status() == _native.ATTN_ERR_DEVICE_ARG
        assert o[1].isfinite().all()
    o, lse = _run(q, pools, scales, table, [-3, 200], 0.09, 128)
    assert _native.attn_get_device_status() == _native.ATTN_ERR_DEVICE_ARG
    assert o[0].abs().max() == 0 and (lse[0] == -float("inf")).all()
    _run(q, pools, scales, table, [100000, 200], 0.09, 128)
    assert _native.attn_get_device_status() == _native.ATTN_ERR_DEVICE_ARG
    assert _native.attn_get_device_status() == 0


def test_far_pages():
    """Pages past 2^31 codes into the pool."""
    page, Hkv, d = 256, 8, 128
    num_pages = 2 ** 31 // (page * Hkv * d) + 3
    table = torch.tensor([[num_pages - 1, 2, num_pages - 2]], dtype=torch.int32)
    lens = [600]
    g, small, scales, t3 = _cache(1, Hkv, d, page, lens, 79, extra=0)
    big = [torch.full((num_pages, page, Hkv, d), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2)]
    bs = [torch.ones((num_pages, Hkv), device="cuda") for _ in range(2)]
    for i in range(2):
        for blk in range(3):
            big[i][table[0, blk]] = small[i][t3[0, blk]].cuda()
            bs[i][table[0, blk]] = scales[i][t3[0, blk]].cuda()
    q = torch.randn((1, 1, 16, d), generator=g).to(torch.bfloat16)
    got = _run(q, big, bs, table, lens, 0.09, 256)
    _check(q, small, scales, t3, lens, 0.09, got, "far pages")


def test_captured_and_two_streams():
    """A captured call replayed, and two calls at once on two streams with workspaces of their own."""
    lens = [900, 400]
    g, pools, scales, table = _cache(2, 2, 128, 64, lens, 80)
    q = torch.randn((2, 1, 8, 128), generator=g).to(torch.bfloat16)
    dev = [q.cuda()] + [p.cuda().view(torch.float8_e4m3fn) for p in pools] + [s.cuda() for s in scales] + [
        table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()]
    want = _native.decode_paged_fp8(*dev, 0.09, 256)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = _native.decode_paged_fp8(*dev, 0.09, 256)
    for _ in range(3):
        graph.replay()
    streams = [torch.cuda.Stream() for _ in range(2)]
    res = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            res.append([_native.decode_paged_fp8(*dev, 0.09, 256) for _ in range(5)])
    torch.cuda.synchronize()
    for o, lse in [got] + res[0] + res[1]:
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    assert _native.attn_get_device_status() == 0


def test_a_late_stream_keeps_what_the_call_allocated():
    """stream=: what the call allocates is that stream's, so allocations of the current stream made while the other
    is still behind do not get its workspace or outputs."""
    lens = [900, 400]
    g, pools, scales, table = _cache(2, 2, 128, 64, lens, 82)
    q = torch.randn((2, 1, 8, 128), generator=g).to(torch.bfloat16)
    dev = [q.cuda()] + [p.cuda().view(torch.float8_e4m3fn) for p in pools] + [s.cuda() for s in scales] + [
        table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()]
    want = _native.decode_paged_fp8(*dev, 0.09, 64)      # 15 splits: partial results in the workspace
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(50_000_000)
    got = _native.decode_paged_fp8(*dev, 0.09, 64, stream=side)
    sizes = [want[0].numel() * 2, want[1].numel() * 4, _native.attn_splitkv_workspace_size(2, 8, 960, 128, 64)]
    held = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(4)]
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert all(bool((h == 255).all()) for h in held)
    assert _native.attn_get_device_status() == 0


def test_refusals():
    lens = [100]
    g, pools, scales, table = _cache(1, 2, 64, 64, lens, 81)
    q = torch.zeros((1, 1, 4, 64), dtype=torch.bfloat16, device="cuda")
    kp, vp = (p.cuda().view(torch.float8_e4m3fn) for p in pools)
    ks, vs = (s.cuda() for s in scales)
    t, n = table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    f = _native.decode_paged_fp8
    for bad in (lambda: f(q.float(), kp, vp, ks, vs, t, n, 0.1), lambda: f(q, kp.view(torch.uint8), vp, ks, vs, t, n, 0.1),
                lambda: f(q, kp, vp, ks[:1], vs, t, n, 0.1), lambda: f(q, kp, vp, ks, vs, t.long(), n, 0.1),
                lambda: f(q, kp, vp, ks, vs, t, n, 0.1, workspace=torch.empty(1 << 20, dtype=torch.uint8)),
                lambda: f(q, kp, vp, ks, vs, t, n, 0.1, workspace=torch.empty(1 << 20, device="cuda")[::2]),
                lambda: f(q, kp, vp, ks, vs, t, n[:0], 0.1), lambda: f(q[:, :, ::2], kp, vp, ks, vs, t, n, 0.1)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: f(q[:, :, :3].contiguous(), kp, vp, ks, vs, t, n, 0.1),
                lambda: f(q, kp, vp, ks, vs, t, n, float("nan")), lambda: f(q, kp, vp, ks, vs, t, n, 0.1, chunk=100),
                lambda: f(q, kp, vp, ks, vs, t, n, 0.1, workspace=torch.empty(16, dtype=torch.uint8, device="cuda")),
                lambda: f(q.expand(1, 65, 4, 64).contiguous(), kp, vp, ks, vs, t, n, 0.1)):
        with pytest.raises(_native.AttnError):
            bad()

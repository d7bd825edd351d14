"""GPU: appending keys and values to a paged cache, bf16 and e4m3, against the
definition in 64 bits; rows that a call does not own stay as they were."""
import math

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


def _bits(t):
    return t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t.view(torch.int16)


class Cache:
    """A paged cache on the CPU with old tokens of every sequence, and its plain 64-bit append."""

    def __init__(self, B, Hkv, d, page, lens, room, fp8, seed):
        self.g = torch.Generator().manual_seed(seed)
        self.B, self.Hkv, self.d, self.page, self.fp8 = B, Hkv, d, page, fp8
        self.lens = torch.tensor(lens, dtype=torch.int32)
        mb = -(-room // page)
        self.num_pages = B * mb + 2
        self.table = torch.randperm(self.num_pages, generator=self.g)[:B * mb].view(B, mb).to(torch.int32)
        shape = (self.num_pages, page, Hkv, d)
        if fp8:  # any codes, stale and free pages' among them (NaN too); scales of all sizes
            self.pools = [torch.randint(0, 256, shape, generator=self.g, dtype=torch.uint8) for _ in range(2)]
            self.scales = [torch.exp2(torch.randint(-12, -3, shape[:1] + (Hkv,), generator=self.g).float())
                           for _ in range(2)]
            for b in range(B):  # valid rows hold numbers
                for blk in range(-(-lens[b] // page)):
                    for pool in self.pools:
                        x = pool[self.table[b, blk]][:max(0, lens[b] - blk * page)]
                        x[(x & 0x7F) == 0x7F] = 0x3C
        else:
            self.pools = [torch.randn(shape, generator=self.g).to(torch.bfloat16) for _ in range(2)]
            self.scales = []

    def gpu(self):
        p = [x.cuda() for x in self.pools]
        if self.fp8:
            p = [x.view(torch.float8_e4m3fn) for x in p]
        return p + [s.cuda() for s in self.scales]

    def want(self, k, v, rope, inter, new):
        """(values, error bounds, which rows are new) of both pools after the call, values in 64 bits (codes, for
        e4m3, as the numbers they are), and the scales."""
        out = []
        for t, (x, pool) in enumerate(zip((k, v), self.pools)):
            val = (pool.view(torch.float8_e4m3fn) if self.fp8 else pool).double()
            err = torch.zeros_like(val)
            mine = torch.zeros(val.shape[:2], dtype=torch.bool)
            sc = self.scales[t].double().clone() if self.fp8 else None
            for b in range(self.B):
                n, L = int(new[b]), int(self.lens[b])
                y = x[b, :n].double()
                slack = torch.zeros_like(y)
                if t == 0 and rope is not None:
                    cs = S.angles(rope, torch.arange(L, L + n))
                    slack = 2.0 ** -22 * y.abs().amax(-1, keepdim=True) + slack   # three fp32 roundings
                    y = S.rotate(y, *cs, inter)
                for blk in range(L // self.page, -(-(L + n) // self.page) if n else 0):
                    pg = int(self.table[b, blk])
                    lo, hi = max(L, blk * self.page), min(L + n, (blk + 1) * self.page)
                    r, m = lo - blk * self.page, hi - lo
                    yy, ss = y[lo - L:hi - L], slack[lo - L:hi - L]
                    if self.fp8:
                        fin = torch.where(yy.isfinite(), yy.abs(), torch.zeros_like(yy))
                        now = S.scale_for(fin.amax(dim=(0, 2)))
                        if r > 0:
                            now = torch.maximum(now, sc[pg])
                            val[pg, :r] = S.round_e4m3(val[pg, :r] * (sc[pg] / now)[:, None])
                        sc[pg] = now
                        yy, ss = yy / now[:, None], ss / now[:, None]
                        val[pg, r:r + m] = torch.where(yy.isfinite(), yy, torch.full_like(yy, float("nan")))
                        err[pg, r:r + m] = torch.maximum(2.0 ** -4 * yy.abs(), torch.tensor(2.0 ** -10).double()) + ss
                    else:
                        val[pg, r:r + m] = yy
                        err[pg, r:r + m] = (2.0 ** -8 * yy.abs() if t == 0 and rope is not None else 0) + ss
                    mine[pg, r:r + m] = True
            out.append((val, err, mine, sc))
        return out


def _run(c, k, v, rope, inter, new=None, out=False, strided=False):
    pools = c.gpu()
    B, Nn, Hkv, d = k.shape
    if strided:
        kv = torch.cat((k, v), 2).cuda()
        kc, vc = kv[:, :, :Hkv], kv[:, :, Hkv:]
    else:
        kc, vc = k.cuda(), v.cuda()
    r = None if rope is None else (rope[0].cuda(), rope[1].cuda())
    after = torch.full((B,), -7, dtype=torch.int32, device="cuda") if out else None
    f = _native.kvcache_append_paged_fp8 if c.fp8 else _native.kvcache_append_paged
    f(kc, vc, *pools, c.table.cuda(), c.lens.cuda(), rope=r, interleaved=inter,
      new_lens=None if new is None else torch.tensor(new, dtype=torch.int32).cuda(), seqlens_out=after)
    return pools, after


def _check(c, k, v, rope, inter, new, pools):
    n = new if new is not None else [k.shape[1]] * c.B
    for t, (val, err, mine, sc) in enumerate(c.want(k, v, rope, inter, n)):
        got = pools[t].cpu()
        num = got.double() if not c.fp8 else got.float().double()
        what = "kv"[t]
        nan = val.isnan()
        assert torch.equal(num.isnan(), nan), what
        ok = (num - val).abs() <= err
        assert (ok | nan).all(), "%s: %d values off" % (what, int((~(ok | nan)).sum()))
        if c.fp8:
            assert torch.equal(pools[2 + t].cpu().double(), sc), what + " scales"
            touched = mine.any(1)
        else:
            touched = torch.zeros(mine.shape[0], dtype=torch.bool)
        # pages that the call does not write to keep every bit; so do, in those it does, the rows behind the new ones
        same = _bits(got) == _bits(c.gpu()[t].cpu())
        keep = ~mine
        if c.fp8:
            for pg in touched.nonzero()[:, 0].tolist():
                keep[pg, :int(mine[pg].nonzero()[0, 0])] = False   # older rows: compared above as numbers
        assert same[keep].all(), what + ": a row that is not the call's changed"


CASES = [
    # B, Hkv, d, page, lens, Nn, new, rot, inter
    (1, 1, 64, 64, [0], 1, None, 64, False),
    (4, 8, 128, 256, [0, 1, 255, 256], 1, None, 128, False),
    (5, 3, 64, 64, [63, 64, 65, 0, 127], 1, None, 32, True),
    (3, 2, 128, 64, [0, 30, 200], 131, [131, 100, 1], 128, False),
    (3, 4, 64, 192, [5, 191, 0], 400, [400, 0, 377], 64, True),
    (2, 5, 128, 256, [100, 255], 300, None, 48, False),
    (2, 1, 64, 512, [511, 3], 700, [600, 700], 0, False),
    (2, 9, 128, 128, [17, 0], 33, [2, 33], 16, True),
    (1, 2, 128, 1024, [700], 500, None, 128, True),
    (2, 1, 128, 1024, [3, 1000], 1500, [1500, 30], 64, False),   # more new rows of a page than a block keeps
    (2, 3, 128, 256, [250, 130], 260, [260, 9], 128, True),      # pages full and nearly empty
    (2, 2, 64, 1024, [1, 1023], 1100, None, 64, False),
    (3, 2, 128, 512, [500, 0, 40], 17, [17, 1, 9], 32, False),
    (2, 1, 128, 320, [319, 100], 333, [320, 333], 128, False),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("B,Hkv,d,page,lens,Nn,new,rot,inter", CASES)
def test_append(fp8, B, Hkv, d, page, lens, Nn, new, rot, inter):
    c = Cache(B, Hkv, d, page, lens, max(lens) + Nn, fp8, 300 + Nn + d + page)
    k, v = (torch.randn((B, Nn, Hkv, d), generator=c.g).to(torch.bfloat16) for _ in range(2))
    rope = _native.rope_table(max(lens) + Nn, rot, device="cpu") if rot else None
    pools, after = _run(c, k, v, rope, inter, new, out=True, strided=True)
    assert _native.attn_get_device_status() == 0
    _check(c, k, v, rope, inter, new, pools)
    n = new if new is not None else [Nn] * B
    assert after.tolist() == [a + b for a, b in zip(lens, n)]


@pytest.mark.parametrize("was", [0.3, 1.0 / 448, 0.75 * 2.0 ** -9, 1.9e-31, 3e-38, 1e-41, 0.0])
@pytest.mark.parametrize("rot", [0, 64])
def test_pages_with_scales_that_are_no_powers_of_two(was, rot):
    """A page written elsewhere, its scale any number: the append takes the next power of two (2^-100 at least) for it,
    multiplies the older codes by the quotient and rounds them once, and rounds the new values once."""
    page, Hkv, d, Nn, lens = 64, 2, 64, 20, [10, 63]
    c = Cache(2, Hkv, d, page, lens, 128, True, 19)
    for s in c.scales:
        s.fill_(was)
    before = float(c.scales[0][0, 0])                      # as fp32 holds it
    size = max(before, 2.0 ** -99)
    k, v = ((torch.randn((2, Nn, Hkv, d), generator=c.g) * 60 * size).to(torch.bfloat16) for _ in range(2))
    rope = _native.rope_table(200, rot, device="cpu") if rot else None
    pools, _ = _run(c, k, v, rope, False)
    assert _native.attn_get_device_status() == 0
    up = 2.0 ** max(-100, math.ceil(math.log2(before)) if before else -100)
    for t, x in enumerate((k, v)):
        got, sc = pools[t].float().double().cpu(), pools[2 + t].double().cpu()
        for b, L in enumerate(lens):
            pg, m = int(c.table[b, 0]), min(Nn, page - L)
            y = x[b, :m].double()
            slack = torch.zeros((m, Hkv, 1), dtype=torch.float64)
            if t == 0 and rot:
                slack = 2.0 ** -22 * y.abs().amax(-1, keepdim=True)    # three fp32 roundings
                y = S.rotate(y, *S.angles(rope, torch.arange(L, L + m)), False)
            now = S.scale_for(y.abs().amax(dim=(0, 2))).clamp(min=up)
            assert torch.equal(sc[pg], now)
            # one rounding to e4m3 of a product that fp32 holds to 2^-24 of it
            old = c.pools[t].view(torch.float8_e4m3fn).double()[pg, :L] * (before / now)[:, None]
            err = torch.clamp(2.0 ** -4 * old.abs(), min=2.0 ** -10) * (1 + 2.0 ** -19)
            assert ((got[pg, :L] - old).abs() <= err).all(), "older rows"
            y, slack = y / now[:, None], slack / now[:, None]
            err = torch.clamp(2.0 ** -4 * y.abs(), min=2.0 ** -10) + slack
            assert ((got[pg, L:L + m] - y).abs() <= err).all(), "new rows"


@pytest.mark.parametrize("grow", [1.0, 3.0, 1000.0, 1e30])
def test_scales_are_raised(grow):
    """Tokens one at a time into the same page, each `grow` times the last at first: the scale rises when it must and
    the older codes follow; twice the same call changes nothing more."""
    page, Hkv, d = 64, 2, 64
    c = Cache(2, Hkv, d, page, [0, 10], page, True, 17)
    for step in range(6):
        k, v = (torch.randn((2, 1, Hkv, d), generator=c.g) * 1e-3 for _ in range(2))
        k, v = ((x * (grow if step == 3 else 1.0)).to(torch.bfloat16) for x in (k, v))
        pools, _ = _run(c, k, v, None, False)
        _check(c, k, v, None, False, None, pools)
        f = _native.kvcache_append_paged_fp8
        again = [p.clone() for p in pools]
        f(k.cuda(), v.cuda(), *again, c.table.cuda(), c.lens.cuda())
        assert all(torch.equal(a.view(torch.uint8) if a.dtype != torch.float32 else a,
                               b.view(torch.uint8) if b.dtype != torch.float32 else b) for a, b in zip(pools, again))
        c.pools = [p.view(torch.uint8).cpu() for p in pools[:2]]
        c.scales = [s.cpu() for s in pools[2:]]
        c.lens += 1
    assert _native.attn_get_device_status() == 0


def test_values_at_the_ends_of_the_range():
    """Zeros, the smallest and largest bf16 values, values on the scale's border, NaN and infinities."""
    page, Hkv, d = 64, 1, 64
    rows = [torch.zeros(d), torch.full((d,), 1e-38), torch.full((d,), 3.38e38), torch.full((d,), 448.0),
            torch.full((d,), 450.0), torch.full((d,), 9.2e-41)]
    for i, row in enumerate(rows):
        c = Cache(1, Hkv, d, page, [0], page, True, 40 + i)
        k = row.view(1, 1, 1, d).to(torch.bfloat16)
        k2 = k.clone()
        k2[..., 3] = float("nan")
        k2[..., 9] = float("-inf")
        pools, _ = _run(c, k, k2, None, False)
        _check(c, k, k2, None, False, None, pools)
    assert _native.attn_get_device_status() == 0


@pytest.mark.parametrize("page,Nn,d", [(256, 256, 128), (512, 300, 64), (64, 40, 128), (1024, 1024, 128)])
def test_one_large_value_and_infinities_anywhere_in_a_page(page, Nn, d):
    """The largest value sits in any thread's share of the page; infinities are left out of the scale, wherever."""
    for at in (0, Nn // 3, Nn - 1):
        c = Cache(1, 2, d, page, [0], 2 * page, True, 50 + at)
        k, v = (torch.randn((1, Nn, 2, d), generator=c.g) for _ in range(2))
        k[0, at, 0, 7] = 1000.0
        v[0, at, 1, d - 1] = -3000.0
        k, v = k.to(torch.bfloat16), v.to(torch.bfloat16)
        rope = _native.rope_table(Nn, 32, device="cpu")
        pools, _ = _run(c, k, v, rope, False)
        _check(c, k, v, rope, False, None, pools)
        v[0, (at + 5) % Nn, 0, 3] = float("inf")
        k[0, (at + 9) % Nn, 1, 40] = float("-inf")     # not among the rotated ones
        pools, _ = _run(c, k, v, rope, False)
        _check(c, k, v, rope, False, None, pools)
    assert _native.attn_get_device_status() == 0


def test_rounding_to_nearest_after_rotation():
    """Rotated values at and next to the codes' ties and the scale's border: angles of 0 (the values as they are) and
    of 45 degrees, every code equal to the one that the fp32 rotation rounds to."""
    d, Nn = 64, 64
    base = torch.tensor([1.0, 1.0625, 1.1875, 1.3125, 1.75, 1.7578125, 1.765625, 1.9375])
    x = (base[:, None] * torch.exp2(torch.arange(-7, 9).float())[None]).reshape(-1)     # 128 values to 496
    k = x[torch.randint(0, 128, (1, Nn, 1, d), generator=torch.Generator().manual_seed(6))].to(torch.bfloat16)
    c = Cache(1, 1, d, 64, [0], 64, True, 55)
    ang = torch.zeros((64, 32))
    ang[::2] = torch.pi / 4
    ang[1::4] = 1e-7
    rope = (ang.cos(), ang.sin())
    pools, _ = _run(c, k, k, rope, False)
    a, b = k[0, :, 0, :32].float(), k[0, :, 0, 32:].float()
    y = torch.cat((a * rope[0] - b * rope[1], b * rope[0] + a * rope[1]), -1)
    s = S.scale_for(y.abs().max().double()).float()
    pg = int(c.table[0, 0])
    assert pools[2][pg, 0].item() == s
    assert torch.equal(pools[0][pg, :, 0].cpu().view(torch.uint8), (y / s).to(torch.float8_e4m3fn).view(torch.uint8))


def test_bad_lengths_pages_and_positions_are_reported():
    """What only the device can see is reported and writes nothing outside: rows past the table, negative lengths,
    pages outside the pool, positions past the tables."""
    page, Hkv, d = 64, 2, 64
    for fp8 in (False, True):
        c = Cache(3, Hkv, d, page, [0, 60, 5], 2 * page, fp8, 60)
        k, v = (torch.randn((3, 100, Hkv, d), generator=c.g).to(torch.bfloat16) for _ in range(2))
        c.lens = torch.tensor([0, 60, 100], dtype=torch.int32)      # 100 + 100 rows: 128 fit
        pools, after = _run(c, k, v, None, False, out=True)
        assert _native.attn_get_device_status() == _native.ATTN_ERR_DEVICE_ARG
        assert after.tolist() == [100, 128, 128]
        _check(c, k, v, None, False, [100, 68, 28], pools)
        c.lens = torch.tensor([-5, 999, 3], dtype=torch.int32)
        pools, after = _run(c, k, v, None, False, out=True)
        assert _native.attn_get_device_status() == _native.ATTN_ERR_DEVICE_ARG
        assert after.tolist() == [100, 128, 103]
        c.lens = torch.tensor([0, 128, 3], dtype=torch.int32)
        _check(c, k, v, None, False, [100, 0, 100], pools)
        # a page outside the pool: its rows are dropped, the others written
        good = c.table.clone()
        for bad in (-1, c.num_pages, 2 ** 31 - 1):
            c.table = good.clone()
            c.table[0, 1] = bad
            pools, _ = _run(c, k, v, None, False, [70, 0, 100])
            assert _native.attn_get_device_status() == _native.ATTN_ERR_DEVICE_ARG
            c.table = good
            _check(c, k, v, None, False, [64, 0, 100], pools)
        # too few table rows: the last one's angles
        rope = _native.rope_table(50, 64, device="cpu")
        pools, _ = _run(c, k, v, rope, False)
        assert _native.attn_get_device_status() == _native.ATTN_ERR_DEVICE_ARG
        wide = tuple(torch.cat((t, t[-1:].expand(200, -1))).contiguous() for t in rope)
        _check(c, k, v, wide, False, [100, 0, 100], pools)
        new = [-1, 500, 0]
        pools, after = _run(c, k, v, None, False, new, out=True)
        assert _native.attn_get_device_status() == _native.ATTN_ERR_DEVICE_ARG
        assert after.tolist() == [0, 128, 3]
    assert _native.attn_get_device_status() == 0


def test_nothing_to_append():
    c = Cache(2, 2, 64, 64, [3, 64], 128, True, 70)
    k = torch.zeros((2, 0, 2, 64), dtype=torch.bfloat16)
    for fp8 in (True, False):
        c = Cache(2, 2, 64, 64, [3, 64], 128, fp8, 70)
        pools, after = _run(c, k, k, None, False, out=True)
        assert after.tolist() == [3, 64]
        _check(c, k, k, None, False, [0, 0], pools)


@pytest.mark.parametrize("fp8", [False, True])
def test_far_pages(fp8):
    """Pages past 2^31 elements into the pool: offsets of 64 bits."""
    page, Hkv, d = 256, 8, 128
    num_pages = 2 ** 31 // (page * Hkv * d) + 3
    dtype = torch.uint8 if fp8 else torch.bfloat16
    pools = [torch.zeros((num_pages, page, Hkv, d), dtype=dtype, device="cuda") for _ in range(2)]
    scales = [torch.zeros((num_pages, Hkv), device="cuda") for _ in range(2)]
    table = torch.tensor([[num_pages - 1, 0, num_pages - 2]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([250], dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v = (torch.randn((1, 400, Hkv, d), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    if fp8:
        _native.kvcache_append_paged_fp8(k, v, *(p.view(torch.float8_e4m3fn) for p in pools), *scales, table, lens)
        pools = [p.view(torch.float8_e4m3fn) for p in pools]
    else:
        _native.kvcache_append_paged(k, v, *pools, table, lens)
    assert _native.attn_get_device_status() == 0
    for x, pool, sc in zip((k, v), pools, scales):
        for lo, pg, r in ((0, num_pages - 1, 250), (6, 0, 0), (262, num_pages - 2, 0)):
            m = min(400 - lo, page - r)
            got = pool[pg, r:r + m].float()
            want = x[0, lo:lo + m].float()
            if fp8:
                got = got * sc[pg][:, None]
                assert ((got - want).abs() <= torch.maximum(2.0 ** -4 * want.abs(), 2.0 ** -10 * sc[pg][:, None])).all()
            else:
                assert torch.equal(got, want)


def test_refusals():
    c = Cache(1, 2, 64, 64, [3], 128, True, 80)
    kp, vp, ks, vs = c.gpu()
    t, n = c.table.cuda(), c.lens.cuda()
    x = torch.zeros((1, 1, 2, 64), dtype=torch.bfloat16, device="cuda")
    f = _native.kvcache_append_paged_fp8
    for bad in (lambda: f(x.float(), x, kp, vp, ks, vs, t, n), lambda: f(x, x, kp.view(torch.uint8), vp, ks, vs, t, n),
                lambda: f(x, x, kp, vp[:2], ks, vs, t, n), lambda: f(x, x, kp, vp, ks.double(), vs, t, n),
                lambda: f(x, x, kp, vp, ks, vs, t.long(), n), lambda: f(x, x, kp, vp, ks, vs, t, n.long()),
                lambda: f(x, x[:, :, :1], kp, vp, ks, vs, t, n), lambda: f(x, x, kp, vp, ks, vs, t.cpu(), n),
                lambda: _native.kvcache_append_paged(x, x, kp, vp, t, n)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(_native.AttnError):
        f(x, x, kp, vp, ks, vs, t, n, seqlens_out=n)      # the lengths before are still being read

"""Plain 64-bit forms of the operators around the attention kernels, and the
error bounds that the tests hold the kernels to.

Bounds.  A rounding to a type is off by at most half a step: bf16 2^-8 of the
value, e4m3 2^-4 of it (2^-10 below its smallest normal value, 2^-6), fp32
2^-24.  Sums in fp32 add up to one such rounding of a partial sum for each
addition.  Each function below says which it counts.
"""
import torch

BORDER = 448.5


def rotate(x, cos, sin, inter, back=False):
    """x [..., d] in 64 bits; cos, sin [..., rot / 2] broadcast over x's heads."""
    rot = 2 * cos.shape[-1]
    x = x.clone()
    i = torch.arange(rot // 2)
    a, b = (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)
    xa, xb = x[..., a], x[..., b]
    sin = -sin if back else sin
    x[..., a], x[..., b] = xa * cos - xb * sin, xb * cos + xa * sin
    return x


def angles(rope, positions):
    """cos, sin [..., 1, rot / 2] in 64 bits at the positions; None without rotation."""
    if rope is None:
        return None
    return tuple(t.double()[positions.long()][..., None, :] for t in rope)


def norm_rope(x, w, eps, cs, inter):
    """(y, size): the result and, for each row, the largest magnitude before the rotation."""
    x = x.double()
    if w is not None:
        x = x * (x.square().mean(-1, keepdim=True) + eps).rsqrt() * w.double()
    size = x.abs().amax(-1, keepdim=True)
    return (x if cs is None else rotate(x, *cs, inter)), size


def norm_rope_bwd(dy, x, w, eps, cs, inter):
    """(dx, bound on its fp32 error, dw, sum of magnitudes of dw's terms)."""
    u = dy.double() if cs is None else rotate(dy.double(), *cs, inter, back=True)
    if w is None:
        return u, 2.0 ** -20 * u.abs().amax(-1, keepdim=True), None, None
    x, w = x.double(), w.double()
    r = (x.square().mean(-1, keepdim=True) + eps).rsqrt()
    xr, g = x * r, u * w
    dx = r * (g - xr * (g * xr).mean(-1, keepdim=True))
    # under 64 roundings of 2^-24 on the two parts of dx
    err = 2.0 ** -18 * r * (g.abs().amax(-1, keepdim=True)
                            + xr.abs().amax(-1, keepdim=True) * (g * xr).abs().mean(-1, keepdim=True))
    t = (u * xr).reshape(-1, x.shape[-1])
    return dx, err, t.sum(0), t.abs().sum(0)


def round_e4m3(x):
    """x (64 bits) to the nearest e4m3 value, ties to even."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(e - 3)
    return torch.round(x / step) * step


def scale_for(amax):
    """The smallest power of two s with amax <= 448.5 s, at least 2^-100."""
    e = torch.floor(torch.log2((amax / BORDER).clamp(min=2.0 ** -101))).clamp(min=-100)
    s = torch.exp2(e)
    return torch.where(amax > BORDER * s, 2 * s, s)


def paged_rows(pool, table, n):
    """The first n rows of each sequence's pages, [B, n, ...], from a pool [num_pages, page_size, ...]."""
    B = table.shape[0]
    return pool[table.long()].reshape((B, -1) + tuple(pool.shape[2:]))[:, :n]


def codes64(pool):
    return pool.view(torch.uint8).clone().view(torch.float8_e4m3fn).double() if pool.dtype == torch.float8_e4m3fn \
        else pool.double()


def decode(q, k, v, lens, scale):
    """Attention of the last Nq tokens in 64 bits.  q [B,Nq,Hq,d]; k, v [B,n,Hkv,d] (what lies behind a sequence's
    end is not looked at).  Returns o, lse and the bounds on their errors before o's rounding to bf16:
      scores: fp32 sums of d products in any order, truncated at worst (2^-23 an addition): ds;
      weights: rounded to 9 bits or more (2^-9 of each), shifted by the scores' error (2 ds): on sum p |v|;
      2^-20 of the largest value for what the rest rounds."""
    B, Nq, Hq, d = q.shape
    Hkv = k.shape[2]
    G = Hq // Hkv
    o = torch.zeros((B, Nq, Hq, d), dtype=torch.float64)
    lse = torch.full((B, Hq, Nq), -float("inf"), dtype=torch.float64)
    eo, el = torch.zeros_like(o), torch.zeros_like(lse)
    for b in range(B):
        for h in range(Hq):
            for i in range(Nq):
                n = int(lens[b]) - Nq + 1 + i
                if n <= 0:
                    continue
                kk, vv, qq = k[b, :n, h // G].double(), v[b, :n, h // G].double(), q[b, i, h].double()
                s = scale * (kk @ qq)
                p = torch.softmax(s, 0)
                o[b, i, h], lse[b, h, i] = p @ vv, torch.logsumexp(s, 0)
                ds = 2.0 ** -23 * d * abs(scale) * float((kk.abs() @ qq.abs()).max())
                eo[b, i, h] = (2.0 ** -9 + 2 * ds) * (p @ vv.abs()) + 2.0 ** -20 * float(vv.abs().max())
                el[b, h, i] = ds + 2.0 ** -20 * (1 + abs(float(lse[b, h, i])))
    return o, lse, eo, el


def assert_within(got, want, bound, what):
    got = got.double().cpu()
    bad = ~((got - want).abs() <= bound)
    assert not bad.any(), "%s: %d of %d values outside their bound, the first at %s: %g, want %g +- %g" % (
        what, int(bad.sum()), bad.numel(), tuple(bad.nonzero()[0].tolist()), got[bad][0], want[bad][0],
        (bound + torch.zeros_like(want))[bad][0])

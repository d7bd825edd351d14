"""Workloads of the serving and training operators around the attention kernels.

Three operators, each in its plain form (elementary torch operations) and as
the framework's own calls:

  qk     norms of queries and keys for each head with the position rotation
         in the same pass, forward and backward
  append keys and values of new tokens into a paged cache, keys rotated on
         the way; bf16 cache, or e4m3 with one scale for each page and head
  decode attention of one or a few new tokens over the paged e4m3 cache

Layouts are the framework's: tensors [B, N, H, d], page pools [num_pages,
page_size, Hkv, d], block tables [B, max_blocks], cache lengths int32 [B].
The scale of a page and head is a power of two, the smallest that brings its
largest value to 448.5 or less (which rounds to 448, the type's largest; the
border is no bf16 value, so none sits on it), at least 2^-100; a page that a
call continues keeps its scale or has it raised, its older codes rounded again.
"""
import math

import torch

own = False

BORDER = 448.5
MIN_EXP = -100  # exponent of the smallest scale


# --------------------------------------------------------------------------- cases
def listed():
    return [
        # the serving decode batch of this repository (16 sequences of 1024 to 16384 keys, 32 query heads on
        # 8 KV heads, 256-key pages), its cache held in 8 bits
        dict(name="decode_serving_batch", op="decode", B=16, Nq=1, Hq=32, Hkv=8, d=128, page=256, lo=1024, hi=16384),
        # one user alone with a short conversation: latency
        dict(name="decode_one_short", op="decode", B=1, Nq=1, Hq=32, Hkv=8, d=128, page=64, lo=701, hi=701),
        # two long documents
        dict(name="decode_long", op="decode", B=2, Nq=1, Hq=32, Hkv=8, d=128, page=256, lo=250001, hi=262144),
        # a few drafted tokens checked at once, small heads, ragged lengths, pages that end inside a key tile
        dict(name="decode_drafted_d64", op="decode", B=24, Nq=3, Hq=24, Hkv=4, d=64, page=192, lo=3, hi=4801),
        # one decode step's new token of each sequence, bf16 cache: latency
        dict(name="append_token_bf16", op="append", B=16, Nn=1, Hkv=8, d=128, page=256, lo=1, hi=4000, bits=16,
             rot=128, inter=False),
        # the same for a larger batch and the 8-bit cache: scales kept or raised
        dict(name="append_token_e4m3", op="append", B=64, Nn=1, Hkv=8, d=128, page=256, lo=1, hi=4000, bits=8,
             rot=128, inter=False),
        # prompts behind a shared prefix, padded to the longest, 8-bit cache
        dict(name="append_prompt_e4m3", op="append", B=8, Nn=8191, Hkv=8, d=128, page=256, lo=0, hi=1000, bits=8,
             rot=128, inter=False),
        # chunks of prompts into a bf16 cache, part of each head rotated, pairs side by side
        dict(name="append_prompt_bf16", op="append", B=5, Nn=2500, Hkv=4, d=64, page=64, lo=0, hi=777, bits=16,
             rot=32, inter=True),
        # a decode step's queries and keys: latency
        dict(name="qk_token", op="qk", B=64, N=1, Hq=32, Hkv=8, d=128, rot=128, inter=False, grad=False),
        # the training shape (4 sequences of 4096), grouped heads, forward
        dict(name="qk_train", op="qk", B=4, N=4096, Hq=32, Hkv=8, d=128, rot=128, inter=False, grad=False),
        # and its backward pass
        dict(name="qk_train_grad", op="qk", B=4, N=4096, Hq=32, Hkv=8, d=128, rot=128, inter=False, grad=True),
        # backward at odd sizes, small heads, part of each head rotated, pairs side by side
        dict(name="qk_odd_grad_d64", op="qk", B=3, N=1001, Hq=9, Hkv=3, d=64, rot=32, inter=True, grad=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "append", "qk"])
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    G = rng.choice([1, 2, 4, 5, 7, 8, 16])
    if op == "decode":
        Nq = rng.choice([1, 1, 1, 2, 4, 7])
        most = min(400000, 10 ** 8 // (Nq * Hkv * G))  # keys of all sequences together
        hi = _log(rng, 1, min(100000, most))
        B = _log(rng, 1, max(1, min(64, most // hi)))
        return dict(op=op, B=B, Nq=Nq, Hq=Hkv * G, Hkv=Hkv, d=d,
                    page=64 * rng.choice([1, 2, 3, 4, 8]), lo=max(1, hi // rng.choice([1, 2, 16])), hi=hi)
    if op == "append":
        Nn = _log(rng, 1, 8191)
        B = _log(rng, 1, max(1, min(64, 32000 // Nn)))
        lo = rng.choice([0, 1, 100])
        return dict(op=op, B=B, Nn=Nn, Hkv=Hkv, d=d, page=64 * rng.choice([1, 2, 3, 4, 8]), lo=lo,
                    hi=lo + _log(rng, 1, 4000), bits=rng.choice([8, 16]), rot=rng.choice([0, 32, d // 2, d]),
                    inter=rng.random() < 0.5)
    N = _log(rng, 1, 8191)
    B = _log(rng, 1, max(1, min(64, 16384 // N)))
    return dict(op=op, B=B, N=N, Hq=Hkv * min(G, 32 // Hkv), Hkv=Hkv, d=d, rot=rng.choice([0, 32, d // 2, d]),
                inter=rng.random() < 0.5, grad=rng.random() < 0.5)


# --------------------------------------------------------------------------- inputs
def _rope_angles(max_pos, rot, device):
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=device) / max(rot, 1))
    return torch.arange(max_pos, dtype=torch.float64, device=device)[:, None] * inv


def _scale_exp(amax):
    """Exponent of the scale of largest values `amax`."""
    m, e = torch.frexp(amax)
    e = torch.where(m > BORDER / 512, e - 8, e - 9)
    return torch.where(amax > 0, e, torch.full_like(e, MIN_EXP)).clamp(min=MIN_EXP)


def _pow2(e):
    """2^e in 32 bits, exactly (e in [-126, 127])."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _pool8(gen, num_pages, page, H, d, spread):
    """A pool of e4m3 pages and its scales: normal values of a size that varies by head and channel."""
    dev = gen.device
    amp = torch.exp(spread * torch.randn((1, 1, H, d), generator=gen, device=dev))
    codes = torch.empty((num_pages, page, H, d), dtype=torch.float8_e4m3fn, device=dev)
    exps = torch.empty((num_pages, H), dtype=torch.int32, device=dev)
    step = max(1, (1 << 26) // (page * H * d))
    for p in range(0, num_pages, step):
        x = torch.randn((min(step, num_pages - p), page, H, d), generator=gen, device=dev) * amp
        e = _scale_exp(x.abs().amax(dim=(1, 3)))
        exps[p:p + step] = e
        codes[p:p + step] = (x * _pow2(-e)[:, None, :, None]).to(torch.float8_e4m3fn)
    return codes, _pow2(exps)


def _bf16(gen, shape, amp=1.0):
    x = torch.empty(shape, dtype=torch.bfloat16, device=gen.device)
    x.normal_(generator=gen)
    return x.mul_(amp) if amp != 1.0 else x


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dev = gen.device
    B, d = c["B"], c["d"]
    if c["op"] == "qk":
        N, Hq, Hkv = c["N"], c["Hq"], c["Hkv"]
        # q and k as a fused projection leaves them: q, k and v heads side by side in a token's row
        c["qkv"] = _bf16(gen, (B, N, Hq + 2 * Hkv, d))
        c["q"], c["k"] = c["qkv"][:, :, :Hq], c["qkv"][:, :, Hq:Hq + Hkv]
        c["wq"] = 1 + 0.2 * torch.randn(d, generator=gen, device=dev)
        c["wk"] = 1 + 0.2 * torch.randn(d, generator=gen, device=dev)
        start = torch.randint(0, 4000, (B, 1), generator=gen, device=dev)
        c["pos"] = (start + torch.arange(N, device=dev)).to(torch.int32)
        a = _rope_angles(4000 + N, c["rot"], dev)
        c["cos"], c["sin"], c["eps"] = a.cos().float(), a.sin().float(), 1e-6
        if c["grad"]:
            c["dq"], c["dk"] = _bf16(gen, (B, N, Hq, d)), _bf16(gen, (B, N, Hkv, d))
        return c
    page, Hkv = c["page"], c["Hkv"]
    lens = torch.randint(c["lo"], c["hi"] + 1, (B,), generator=gen, device=dev)
    if c["op"] == "decode":
        lens = lens.clamp(min=c["Nq"])
        cap = max(c["hi"], c["Nq"])
    else:
        cap = c["hi"] + c["Nn"]
    blocks = -(-cap // page)
    num_pages = B * blocks + 3
    c["table"] = torch.randperm(num_pages, generator=gen, device=dev)[:B * blocks].view(B, blocks).to(torch.int32)
    c["lens"] = lens.to(torch.int32)
    if c["op"] == "decode":
        c["q"] = _bf16(gen, (B, c["Nq"], c["Hq"], d))
        c["kp"], c["ks"] = _pool8(gen, num_pages, page, Hkv, d, 0.25)
        c["vp"], c["vs"] = _pool8(gen, num_pages, page, Hkv, d, 0.25)
        # what lies behind a sequence's end is of no meaning: here it is NaN in its last page
        last = c["table"].gather(1, ((lens - 1) // page)[:, None])[:, 0].long()
        stale = torch.arange(page, device=dev) >= ((lens - 1) % page + 1)[:, None]
        for pool in (c["kp"], c["vp"]):
            u = pool.view(torch.uint8)
            u[last] = torch.where(stale[:, :, None, None], torch.full_like(u[last], 0x7F), u[last])
        c["scale"] = d ** -0.5
        return c
    Nn = c["Nn"]
    # the new tokens as a fused projection leaves them (k and v heads side by side), padded to Nn a sequence
    c["kv"] = _bf16(gen, (B, Nn, 2 * Hkv, d))
    c["kv"].mul_(torch.exp(0.5 * torch.randn((B, Nn, 1, 1), generator=gen, device=dev)).to(torch.bfloat16))
    c["k"], c["v"] = c["kv"][:, :, :Hkv], c["kv"][:, :, Hkv:]
    c["new"] = torch.randint((Nn + 1) // 2, Nn + 1, (B,), generator=gen, device=dev).to(torch.int32)
    a = _rope_angles(cap, c["rot"], dev)
    c["cos"], c["sin"] = a.cos().float(), a.sin().float()
    if c["bits"] == 8:
        c["kp"], c["ks"] = _pool8(gen, num_pages, page, Hkv, d, 0.25)
        c["vp"], c["vs"] = _pool8(gen, num_pages, page, Hkv, d, 0.25)
    else:
        c["kp"], c["vp"] = (_bf16(gen, (num_pages, page, Hkv, d)) for _ in range(2))
    return c


# --------------------------------------------------------------------------- plain forms
def _rotate(x, cos, sin, rot, inter, back=False):
    """Rotation of the first `rot` values of x [..., H, d]; cos, sin [..., 1, rot / 2]; `back`: by the negative angle."""
    if rot == 0:
        return x
    r, rest = x[..., :rot], x[..., rot:]
    a, b = (r[..., 0::2], r[..., 1::2]) if inter else (r[..., :rot // 2], r[..., rot // 2:])
    if back:
        sin = -sin
    p, q = a * cos - b * sin, b * cos + a * sin
    r = torch.stack((p, q), -1).flatten(-2) if inter else torch.cat((p, q), -1)
    return torch.cat((r, rest), -1)


def _plain_qk(s):
    pos = s["pos"].long()
    cos, sin = s["cos"][pos][:, :, None], s["sin"][pos][:, :, None]
    out = []
    for x, w, dy in ((s["q"], s["wq"], s.get("dq")), (s["k"], s["wk"], s.get("dk"))):
        x = x.float()
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"])
        if dy is None:
            out.append(_rotate(x * r * w, cos, sin, s["rot"], s["inter"]).to(torch.bfloat16))
            continue
        du = _rotate(dy.float(), cos, sin, s["rot"], s["inter"], back=True)
        xr = x * r
        g = du * w
        out.append((r * (g - xr * (g * xr).mean(-1, keepdim=True))).to(torch.bfloat16))
        out.append((du * xr).sum((0, 1, 2), dtype=torch.float64).float())
    return out


def _slots(s):
    """(page, row) of each new token [B, Nn]; a padded one has those of its sequence's last token, as its index."""
    i = torch.minimum(torch.arange(s["Nn"], device=s["lens"].device), s["new"].long()[:, None] - 1)
    at = s["lens"].long()[:, None] + i
    return i, at, s["table"].long().gather(1, at // s["page"]), at % s["page"]


def _plain_append(s):
    Nn, page, Hkv, d = s["Nn"], s["page"], s["Hkv"], s["d"]
    i, at, pg, row = _slots(s)
    b = torch.arange(s["B"], device=i.device)[:, None]
    k = _rotate(s["k"][b, i].float(), s["cos"][at][:, :, None], s["sin"][at][:, :, None], s["rot"], s["inter"])
    if s["bits"] == 16:
        s["kp"][pg, row] = k.to(torch.bfloat16)
        s["vp"][pg, row] = s["v"][b, i]
        return s["kp"], s["vp"]
    # the pages that a sequence's new tokens reach, [B, P]; those past its last one repeat it
    first = s["lens"].long() // page
    lastp = (s["lens"].long() + s["new"].long() - 1) // page
    P = (Nn + page - 2) // page + 1
    blk = torch.minimum(first[:, None] + torch.arange(P, device=i.device), lastp[:, None])
    tgt = s["table"].long().gather(1, blk)
    rows = blk[:, :, None] * page + torch.arange(page, device=i.device)  # the position of each row of these pages
    older = rows < s["lens"].long()[:, None, None]
    at_new = (rows - s["lens"].long()[:, None, None]).clamp(0, Nn - 1)
    is_new = ~older & (rows < (s["lens"].long() + s["new"].long())[:, None, None])
    bb = b[:, :, None]
    has_old = older.any(-1)[:, :, None]
    for x, pool, scales in ((k, s["kp"], s["ks"]), (s["v"][b, i].float(), s["vp"], s["vs"])):
        codes = pool.view(torch.uint8)[tgt]
        x = x[bb, at_new]
        amax = torch.where(is_new[..., None, None], x.abs(), torch.zeros_like(x)).amax(dim=(2, 4))
        was = torch.where(has_old, scales[tgt], torch.zeros_like(scales[tgt]))
        now = torch.maximum(was, _pow2(_scale_exp(amax)))
        fresh = (x * (1.0 / now)[:, :, None, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        again = (codes.view(torch.float8_e4m3fn).float() * (was / now)[:, :, None, :, None]).to(torch.float8_e4m3fn)
        codes = torch.where(is_new[..., None, None], fresh,
                            torch.where(older[..., None, None], again.view(torch.uint8), codes))
        pool.view(torch.uint8)[tgt] = codes
        scales[tgt] = now
    return s["kp"], s["vp"], s["ks"], s["vs"]


def _plain_decode(s):
    B, Nq, Hq, Hkv, d, page = (s[n] for n in ("B", "Nq", "Hq", "Hkv", "d", "page"))
    t = s["table"].long()
    n = t.shape[1] * page
    seen = torch.arange(n, device=t.device) <= (s["lens"].long()[:, None] - Nq + torch.arange(Nq, device=t.device)
                                                )[:, :, None]  # [B, Nq, n]
    end = (torch.arange(n, device=t.device) < s["lens"][:, None])[:, None, :, None]
    k, v = (torch.where(end, (pool.view(torch.uint8)[t].view(torch.float8_e4m3fn).float()
                              * sc[t][:, :, None, :, None]).view(B, n, Hkv, d).transpose(1, 2), 0.0)
            for pool, sc in ((s["kp"], s["ks"]), (s["vp"], s["vs"])))  # [B, Hkv, n, d]
    G = Hq // Hkv
    q = s["q"].float().view(B, Nq, Hkv, G, d).permute(0, 2, 1, 3, 4).reshape(B, Hkv, Nq * G, d)
    x = (q @ k.transpose(2, 3)).mul_(s["scale"]).view(B, Hkv, Nq, G, n)
    x = x.masked_fill_(~seen[:, None, :, None, :], -math.inf)
    m = x.amax(-1, keepdim=True)
    p = x.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = (p.view(B, Hkv, Nq * G, n) @ v).view(B, Hkv, Nq, G, d) / l
    lse = (m + l.log())[..., 0]
    return (o.permute(0, 2, 1, 3, 4).reshape(B, Nq, Hq, d).to(torch.bfloat16),
            lse.permute(0, 1, 3, 2).reshape(B, Hq, Nq).contiguous())


def run(s):
    if not own:
        return {"qk": _plain_qk, "append": _plain_append, "decode": _plain_decode}[s["op"]](s)
    from exact_io_aware_14_gb300 import _native as A
    if s["op"] == "qk":
        kw = dict(rope=(s["cos"], s["sin"]) if s["rot"] else None, positions=s["pos"], interleaved=s["inter"])
        if not s["grad"]:
            return A.qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], s["eps"], **kw)
        dq, dk, dwq, dwk = A.qk_norm_rope_bwd(s["dq"], s["dk"], s["q"], s["k"], s["wq"], s["wk"], s["eps"], **kw)
        return [dq, dwq, dk, dwk]
    if s["op"] == "append":
        kw = dict(rope=(s["cos"], s["sin"]) if s["rot"] else None, interleaved=s["inter"], new_lens=s["new"])
        if s["bits"] == 16:
            A.kvcache_append_paged(s["k"], s["v"], s["kp"], s["vp"], s["table"], s["lens"], **kw)
            return s["kp"], s["vp"]
        A.kvcache_append_paged_fp8(s["k"], s["v"], s["kp"], s["vp"], s["ks"], s["vs"], s["table"], s["lens"], **kw)
        return s["kp"], s["vp"], s["ks"], s["vs"]
    return A.decode_paged_fp8(s["q"], s["kp"], s["vp"], s["ks"], s["vs"], s["table"], s["lens"], s["scale"])


# --------------------------------------------------------------------------- work
def work(case):
    """Inputs once, outputs once: bytes; multiplications and additions of the products: flops.  Lengths at their mean."""
    c = case
    B, d = c["B"], c["d"]
    if c["op"] == "qk":
        rows = B * c["N"] * (c["Hq"] + c["Hkv"])
        table = B * c["N"] * c["rot"] * 4
        return {"bytes": rows * d * 2 * (3 if c["grad"] else 2) + table,
                "flops": rows * d * (18 if c["grad"] else 8)}
    if c["op"] == "append":
        tokens = B * ((c["Nn"] + 1) // 2 + c["Nn"]) / 2
        return {"bytes": tokens * (c["Hkv"] * d * 2 * (2 + c["bits"] // 8) + c["rot"] * 4),
                "flops": tokens * c["Hkv"] * d * 8}
    keys = B * max((c["lo"] + c["hi"]) / 2, c["Nq"])
    qo = B * c["Nq"] * c["Hq"] * d * 4
    return {"bytes": keys * c["Hkv"] * (2 * d + 8 / c["page"]) + qo, "flops": 4 * keys * c["Nq"] * c["Hq"] * d}


# --------------------------------------------------------------------------- from the definition, in 64 bits
def _exact_table(c):
    """The rotation as the caller's tables hold it: they are inputs, in 32 bits."""
    return c["cos"].double(), c["sin"].double()


def _exact_pairs(x, cos, sin, rot, inter):
    """x [..., d], the pairs of its first `rot` values taken as complex numbers and multiplied by cos + i sin."""
    x = x.clone()
    if rot:
        i = torch.arange(rot // 2, device=x.device)
        re, im = (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)
        z = torch.complex(x[..., re], x[..., im]) * torch.complex(cos, sin)
        x[..., re], x[..., im] = z.real, z.imag
    return x


def _exact_round8(x):
    """x to the nearest value of e4m3 (ties to even): steps of 2^-9 below 2^-6, of 2^(e-3) in [2^e, 2^(e+1))."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(e - 3)
    return torch.round(x / step) * step


def exact(case, seed):
    c = prepare(case, seed)
    B, d = c["B"], c["d"]
    if c["op"] == "qk":
        cos, sin = _exact_table(c)
        cos, sin = (t[c["pos"].long()][:, :, None] for t in (cos, sin))
        out = []
        for x, w, dy in ((c["q"], c["wq"], c.get("dq")), (c["k"], c["wk"], c.get("dk"))):
            x, w = x.double(), w.double()
            n = (x.square().sum(-1, keepdim=True) / d + c["eps"]).sqrt()
            if dy is None:
                out.append(_exact_pairs(x / n * w, cos, sin, c["rot"], c["inter"]))
                continue
            u = _exact_pairs(dy.double(), cos, -sin, c["rot"], c["inter"])
            out.append(u * w / n - x * (u * w * x).sum(-1, keepdim=True) / (d * n ** 3))
            out.append((u * x / n).reshape(-1, d).sum(0))
        return out
    lens, page = c["lens"].tolist(), c["page"]
    if c["op"] == "append":
        new = c["new"].tolist()
        cos, sin = _exact_table(c)
        k8 = c["bits"] == 8
        pools = [c["kp"].to(torch.float64), c["vp"].to(torch.float64)]
        scales = [c["ks"].double(), c["vs"].double()] if k8 else [None, None]
        for b in range(B):
            at = torch.arange(lens[b], lens[b] + new[b], device=c["k"].device)
            kk = _exact_pairs(c["k"][b, :new[b]].double(), cos[at][:, None], sin[at][:, None], c["rot"], c["inter"])
            for x, pool, sc in zip((kk, c["v"][b, :new[b]].double()), pools, scales):
                for blk in range(lens[b] // page, (lens[b] + new[b] - 1) // page + 1):
                    pg = int(c["table"][b, blk])
                    lo, hi = max(lens[b], blk * page), min(lens[b] + new[b], (blk + 1) * page)
                    y, r = x[lo - lens[b]:hi - lens[b]], lo - blk * page
                    if k8:
                        need = torch.exp2(torch.ceil(torch.log2((y.abs().amax(dim=(0, 2)) / BORDER)
                                                                .clamp(min=2.0 ** MIN_EXP))))
                        now = torch.maximum(need, sc[pg]) if r > 0 else need
                        pool[pg, :r] = _exact_round8(pool[pg, :r] * (sc[pg] / now)[:, None])
                        y, sc[pg] = _exact_round8(y / now[:, None]), now
                    pool[pg, r:r + hi - lo] = y
        return pools + scales if k8 else pools
    Nq, Hq, Hkv = c["Nq"], c["Hq"], c["Hkv"]
    G = Hq // Hkv
    o = torch.empty((B, Nq, Hq, d), dtype=torch.float64, device=c["q"].device)
    lse = torch.empty((B, Hq, Nq), dtype=torch.float64, device=c["q"].device)
    for b in range(B):
        pg = c["table"][b, :-(-lens[b] // page)].long()
        for h in range(Hkv):
            k, v = ((pool.view(torch.uint8)[pg, :, h].view(torch.float8_e4m3fn).double() * sc[pg, h].double()[:, None, None]
                     ).reshape(-1, d)[:lens[b]] for pool, sc in ((c["kp"], c["ks"]), (c["vp"], c["vs"])))
            for i in range(Nq):
                n = lens[b] - Nq + 1 + i
                x = c["scale"] * (c["q"][b, i, h * G:(h + 1) * G].double() @ k[:n].T)
                lse[b, h * G:(h + 1) * G, i] = torch.logsumexp(x, -1)
                o[b, i, h * G:(h + 1) * G] = torch.softmax(x, -1) @ v[:n]
    return [o, lse]

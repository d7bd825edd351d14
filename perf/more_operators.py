"""Workloads of the operators that work on a paged cache beyond one decode step.

Five operators, each in its plain form (elementary torch operations) and as
the framework's own calls:

  tables  block tables and slot maps built on the GPU: finished sequences give
          their pages back, the others get pages for their new tokens
  shared  attention of one or a few new tokens of each sequence where the
          batch shares a long prefix, the prefix read once for all
  bounds  the smallest and largest key of each channel in blocks of 64 keys
  select  the blocks whose bounds allow the largest scores, for each query
          and KV head
  attend  attention of each query over the blocks selected for it

Layouts are the framework's: tensors [B, N, H, d], page pools [num_pages,
page_size, Hkv, d], block tables [B, max_blocks], cache lengths int32 [B] with
the new tokens counted (in `tables`: before them).  Block j of a sequence is
its keys 64 j .. 64 j + 63.  The new token n of Nq sits at position
L - Nq + n and sees the keys up to its own.
"""
import math

import torch

own = False

BLOCK = 64


# --------------------------------------------------------------------------- cases
def listed():
    return [
        # a decode step's bookkeeping: some sequences finish, the others take one token each: latency
        dict(name="tables_step", op="tables", B=256, Nn=1, page=64, hi=4000),
        # a batch of prompts comes in, with the slot of each of their tokens
        dict(name="tables_prompts", op="tables", B=48, Nn=8191, page=256, hi=1000),
        # a few chats behind a short instruction: latency
        dict(name="shared_few_short", op="shared", B=4, Nq=1, Hq=32, Hkv=8, d=128, page=64, shared=1024, lo=1, hi=300),
        # many users behind one long document
        dict(name="shared_document", op="shared", B=64, Nq=1, Hq=32, Hkv=8, d=128, page=256, shared=32768, lo=1,
             hi=2048),
        # many samples of one prompt, a few drafted tokens each, small heads, pages that end inside a tile
        dict(name="shared_samples_d64", op="shared", B=96, Nq=3, Hq=24, Hkv=4, d=64, page=192, shared=19200, lo=3,
             hi=601),
        # one decode step's new token of each sequence: latency
        dict(name="bounds_token", op="bounds", B=64, Nn=1, Hkv=8, d=128, page=256, lo=1, hi=4000),
        # prompts, padded to the longest
        dict(name="bounds_prompt", op="bounds", B=8, Nn=8191, Hkv=8, d=128, page=256, lo=0, hi=1000),
        # the decode batch of this repository at longer contexts
        dict(name="select_token", op="select", B=16, Nq=1, Hq=32, Hkv=8, d=128, page=256, lo=16384, hi=131072, topk=64),
        # a chunk of a long prompt
        dict(name="select_prompt", op="select", B=1, Nq=2048, Hq=32, Hkv=8, d=128, page=256, lo=32768, hi=32768,
             topk=32),
        # and the attention over the blocks selected
        dict(name="attend_token", op="attend", B=16, Nq=1, Hq=32, Hkv=8, d=128, page=256, lo=16384, hi=65536, topk=64),
        dict(name="attend_prompt", op="attend", B=1, Nq=2048, Hq=32, Hkv=8, d=128, page=256, lo=32768, hi=32768,
             topk=32),
        # drafted tokens over short and long sequences, odd head counts, small heads: some lists are not full
        dict(name="attend_drafted_d64", op="attend", B=5, Nq=3, Hq=9, Hkv=3, d=64, page=192, lo=3, hi=5000, topk=7),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["tables", "shared", "bounds", "select", "attend"])
    d = rng.choice([64, 128])
    page = 64 * rng.choice([1, 2, 3, 4, 8])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    G = rng.choice([1, 2, 4, 5, 7, 8])
    if op == "tables":
        Nn = _log(rng, 1, 8191)
        return dict(op=op, B=_log(rng, 1, min(1024, 390000 // Nn)), Nn=Nn, page=page, hi=_log(rng, 1, 8000))
    if op == "shared":
        Nq = rng.choice([1, 1, 1, 2, 4, 7])
        B = _log(rng, 1, 128)
        shared = page * (_log(rng, 1, max(1, min(32768, (1 << 29) // (B * Nq * G * Hkv * 8)) // page)) - 1)
        hi = _log(rng, Nq, max(Nq, min(8192, 131072 // B, (1 << 29) // (B * Nq * G * Hkv * 8))))
        return dict(op=op, B=B, Nq=Nq, Hq=Hkv * G, Hkv=Hkv, d=d, page=page, shared=shared,
                    lo=max(1, hi // rng.choice([1, 2, 16])), hi=hi)
    if op == "bounds":
        Nn = _log(rng, 1, 8191)
        B = _log(rng, 1, min(64, 65528 // Nn))
        return dict(op=op, B=B, Nn=Nn, Hkv=Hkv, d=d, page=page, lo=0, hi=_log(rng, 1, 4000))
    Nq = rng.choice([1, 1, 2, 5, _log(rng, 8, 2048)])
    hi = _log(rng, max(Nq, 64), 65536 if Nq < 8 else 32768)
    topk = _log(rng, 3, 64 if Nq < 8 else 32)
    most = (1 << 24) // (Nq * Hkv * G * -(-hi // BLOCK)) if op == "select" else 131072 // (Nq * Hkv * topk)
    B = _log(rng, 1, max(1, min(32, most, (1 << 20) // hi)))
    return dict(op=op, B=B, Nq=Nq, Hq=Hkv * G, Hkv=Hkv, d=d, page=page, lo=max(1, hi // rng.choice([1, 2, 16])),
                hi=hi, topk=topk)


# --------------------------------------------------------------------------- inputs
def _bf16(gen, shape):
    x = torch.empty(shape, dtype=torch.bfloat16, device=gen.device)
    return x.normal_(generator=gen)


def _stale(pools, table, lens, page):
    """What lies behind a sequence's end is of no meaning: here it is NaN in its last page."""
    last = table.long().gather(1, ((lens.long() - 1).clamp(min=0) // page)[:, None])[:, 0]
    behind = torch.arange(page, device=lens.device) >= ((lens.long() - 1) % page + 1)[:, None]
    for pool in pools:
        pool[last] = pool[last].masked_fill(behind[:, :, None, None], math.nan)


def _bounds_of(kp, page):
    """Bounds of all the blocks of a pool, in its layout."""
    n, _, H, d = kp.shape
    x = kp.view(n, page // BLOCK, BLOCK, H, d)
    return torch.stack((x.amin(2), x.amax(2)), 3)


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dev = gen.device
    B, page = c["B"], c["page"]
    if c["op"] == "tables":
        Nn = c["Nn"]
        blocks = -(-(c["hi"] + Nn) // page)
        num = B * blocks + 5
        lens = torch.randint(0, c["hi"] + 1, (B,), generator=gen, device=dev)
        done = torch.rand((B,), generator=gen, device=dev) < 0.1
        new = torch.randint((Nn + 1) // 2, Nn + 1, (B,), generator=gen, device=dev)
        c["lens"] = lens.to(torch.int32)
        c["keep"] = torch.where(done, 0, lens).to(torch.int32)
        c["new"] = torch.where(done, 0, new).to(torch.int32)
        # pages in use are handed out first, what is left is the free list; in half of the seeds it falls short
        pages = torch.randperm(num, generator=gen, device=dev).to(torch.int32)
        used = -(-lens // page)
        first = used.cumsum(0) - used
        col = torch.arange(blocks, device=dev)
        at = first[:, None] + col
        c["table"] = torch.where(col < used[:, None], pages[at.clamp(max=num - 1)], -1).to(torch.int32)
        n_used = used.sum()
        c["num"] = num
        c["free"] = torch.cat((pages, pages))[(n_used + torch.arange(num, device=dev))].contiguous()
        left = num - n_used
        if seed % 2:
            need = torch.where(done, 0, -(-(lens + new) // page) - used).sum()
            left = torch.minimum(left, need * 3 // 4)
        c["count"] = left.to(torch.int32).view(1)
        return c
    if c["op"] == "bounds":
        Hkv, d, Nn = c["Hkv"], c["d"], c["Nn"]
        before = torch.randint(c["lo"], c["hi"] + 1, (B,), generator=gen, device=dev)
        new = torch.randint((Nn + 1) // 2, Nn + 1, (B,), generator=gen, device=dev)
        blocks = -(-(c["hi"] + Nn) // page)
        num = B * blocks + 3
        c["table"] = torch.randperm(num, generator=gen, device=dev)[:B * blocks].view(B, blocks).to(torch.int32)
        c["lens"], c["new"] = (before + new).to(torch.int32), new.to(torch.int32)
        c["kp"] = _bf16(gen, (num, page, Hkv, d))
        _stale((c["kp"],), c["table"], c["lens"], page)
        c["kb"] = torch.zeros((num, page // BLOCK, Hkv, 2, d), dtype=torch.bfloat16, device=dev)
        return c
    Nq, Hq, Hkv, d = c["Nq"], c["Hq"], c["Hkv"], c["d"]
    c["scale"] = d ** -0.5
    lens = torch.randint(c["lo"], c["hi"] + 1, (B,), generator=gen, device=dev).clamp(min=Nq)
    if c["op"] == "shared":
        pre, blocks = c["shared"] // page, -(-max(c["hi"], Nq) // page)
        num = pre + B * blocks + 3
        perm = torch.randperm(num, generator=gen, device=dev).to(torch.int32)
        c["table"] = torch.cat((perm[:pre].expand(B, pre), perm[pre:pre + B * blocks].view(B, blocks)), 1).contiguous()
        lens = lens + c["shared"]
    else:
        blocks = -(-max(c["hi"], Nq) // page)
        num = B * blocks + 3
        c["table"] = torch.randperm(num, generator=gen, device=dev)[:B * blocks].view(B, blocks).to(torch.int32)
    c["lens"] = lens.to(torch.int32)
    c["q"] = _bf16(gen, (B, Nq, Hq, d))
    c["kp"] = _bf16(gen, (num, page, Hkv, d))
    if c["op"] == "select":
        c["kb"] = _bounds_of(c["kp"], page)
        del c["kp"]
        return c
    c["vp"] = _bf16(gen, (num, page, Hkv, d))
    _stale((c["kp"], c["vp"]), c["table"], c["lens"], page)
    if c["op"] == "attend":
        # the query's own block and others of its past, as a selection leaves them: ascending, -1 behind
        pos = lens[:, None] - Nq + torch.arange(Nq, device=dev)
        mine = (pos // BLOCK)[:, :, None, None]
        n = blocks * (page // BLOCK)
        j = torch.arange(n, device=dev)
        key = torch.rand((B, Nq, Hkv, n), generator=gen, device=dev)
        key = key.masked_fill_(j > mine, -1.0).masked_fill_(j == mine, 2.0)
        val, idx = key.topk(min(c["topk"], n), -1)
        idx = torch.where(val < 0, n, idx).sort(-1).values
        idx = torch.where(idx == n, -1, idx).to(torch.int32)
        c["blocks"] = torch.full((B, Nq, Hkv, c["topk"]), -1, dtype=torch.int32, device=dev)
        c["blocks"][..., :idx.shape[-1]] = idx
    return c


# --------------------------------------------------------------------------- plain forms
def _plain_tables(s):
    page, Nn, num = s["page"], s["Nn"], s["num"]
    lens, keep, new, table, free = s["lens"].long(), s["keep"].long(), s["new"].long(), s["table"], s["free"]
    col = torch.arange(table.shape[1], device=lens.device)
    # pages back: the last sequence's last page first
    had, have = -(-lens // page), -(-keep // page)
    back = had - have
    after = back.flip(0).cumsum(0).flip(0) - back
    at = s["count"].long() + after[:, None] + (had[:, None] - 1 - col)
    ok = (col >= have[:, None]) & (col < had[:, None])
    free[at[ok]] = table[ok]
    count = s["count"].long() + back.sum()
    # pages for the new tokens, sequence by sequence while they last
    need = -(-(keep + new) // page) - have
    ends = need.cumsum(0)
    served = (need == 0) | (ends <= count)  # who wants no page gets its tokens in any case
    granted = torch.where(served, new, 0)
    j = (ends - need)[:, None] + (col - have[:, None])
    ok = served[:, None] & (col >= have[:, None]) & (col < (have + need)[:, None])
    table.copy_(torch.where(ok, free[(count - 1 - j).clamp(0, num - 1)], table))
    count2 = count - torch.where(served, need, 0).sum()
    i = torch.arange(Nn, device=lens.device)
    pos = keep[:, None] + i
    slot = table.long().gather(1, (pos // page).clamp(max=table.shape[1] - 1)) * page + pos % page
    return (table, free, granted.to(torch.int32), torch.where(i < granted[:, None], slot, -1),
            count2.to(torch.int32).view(1))


def _plain_shared(s):
    B, Nq, Hq, Hkv, d, page, P = (s[n] for n in ("B", "Nq", "Hq", "Hkv", "d", "page", "shared"))
    G, t = Hq // Hkv, s["table"].long()
    pre = P // page
    n = (t.shape[1] - pre) * page
    pos = s["lens"].long()[:, None] - Nq + torch.arange(Nq, device=t.device)  # [B, Nq]
    end = (P + torch.arange(n, device=t.device) < s["lens"][:, None])[:, :, None, None]
    kc, vc = (s[x][t[0, :pre]].float().view(P, Hkv, d).transpose(0, 1) for x in ("kp", "vp"))  # [Hkv, P, d]
    k, v = (torch.where(end, s[x][t[:, pre:]].view(B, n, Hkv, d).float(), 0.0).transpose(1, 2) for x in ("kp", "vp"))
    q = s["q"].float().view(B, Nq, Hkv, G, d).permute(2, 0, 1, 3, 4).contiguous()  # [Hkv, B, Nq, G, d]
    xc = (q.view(Hkv, -1, d) @ kc.transpose(1, 2)).mul_(s["scale"]).view(Hkv, B, Nq, G, P)
    xo = (q.view(Hkv, B, Nq * G, d).transpose(0, 1) @ k.transpose(2, 3)).mul_(s["scale"]).view(B, Hkv, Nq, G, n)
    xo = xo.transpose(0, 1).masked_fill((P + torch.arange(n, device=t.device) > pos[:, :, None])[:, :, None, :],
                                        -math.inf)
    m = xo.amax(-1, keepdim=True)
    if P:
        m = torch.maximum(m, xc.amax(-1, keepdim=True))
    pc, po = xc.sub_(m).exp_(), xo.sub_(m).exp_()
    l = pc.sum(-1, keepdim=True) + po.sum(-1, keepdim=True)
    o = (pc.view(Hkv, -1, P) @ vc).view(Hkv, B, Nq, G, d)
    o = o + (po.transpose(0, 1).reshape(B, Hkv, Nq * G, n) @ v).view(B, Hkv, Nq, G, d).transpose(0, 1)
    lse = (m + l.log())[..., 0]
    return ((o / l).permute(1, 2, 0, 3, 4).reshape(B, Nq, Hq, d).to(torch.bfloat16),
            lse.permute(1, 0, 3, 2).reshape(B, Hq, Nq).contiguous())


def _plain_bounds(s):
    page, Nn, Hkv, d, B = s["page"], s["Nn"], s["Hkv"], s["d"], s["B"]
    lens, new, t, dev = s["lens"].long(), s["new"].long(), s["table"].long(), s["lens"].device
    # the blocks that a sequence's new tokens reach; those past its last one repeat it
    n = (Nn + BLOCK - 2) // BLOCK + 1
    blk = torch.minimum(((lens - new) // BLOCK)[:, None] + torch.arange(n, device=dev), ((lens - 1) // BLOCK)[:, None])
    pg, sub = t.gather(1, blk * BLOCK // page), blk % (page // BLOCK)
    x = s["kp"].view(-1, page // BLOCK, BLOCK, Hkv, d)[pg, sub].float()  # [B, n, 64, Hkv, d]
    behind = (blk[:, :, None] * BLOCK + torch.arange(BLOCK, device=dev) >= lens[:, None, None])[..., None, None]
    s["kb"][pg, sub] = torch.stack((x.masked_fill(behind, math.inf).amin(2), x.masked_fill(behind, -math.inf).amax(2)),
                                   3).to(torch.bfloat16)
    return s["kb"]


def _plain_select(s):
    B, Nq, Hq, Hkv, d, page, topk = (s[n] for n in ("B", "Nq", "Hq", "Hkv", "d", "page", "topk"))
    G, dev, n = Hq // Hkv, s["q"].device, s["table"].shape[1] * (s["page"] // BLOCK)
    out = torch.full((B, Nq, Hkv, topk), -1, dtype=torch.int32, device=dev)
    j, k = torch.arange(n, device=dev), min(topk, n)
    for b in range(B):
        kb = s["kb"][s["table"][b].long()].view(n, Hkv, 2, d).double()
        q = s["q"][b].double().view(Nq, Hkv, G, d).transpose(0, 1).reshape(Hkv, Nq * G, d)
        # 64 bits: which of two blocks ranks first hangs on the last bits of their scores
        x = q.clamp(min=0) @ kb[:, :, 1].permute(1, 2, 0) + q.clamp(max=0) @ kb[:, :, 0].permute(1, 2, 0)
        x = x.view(Hkv, Nq, G, n).amax(2)
        last = (s["lens"][b].long() - Nq + torch.arange(Nq, device=dev))[:, None] // BLOCK
        x = x.masked_fill_((j < 1) | (j >= last), math.inf).masked_fill_(j > last, -math.inf)
        val, idx = x.sort(dim=-1, descending=True, stable=True)
        idx = torch.where(val[..., :k] == -math.inf, n, idx[..., :k]).sort(-1).values
        out[b, :, :, :k] = torch.where(idx == n, -1, idx).transpose(0, 1).to(torch.int32)
    return out


def _plain_attend(s):
    B, Nq, Hq, Hkv, d, page, topk = (s[n] for n in ("B", "Nq", "Hq", "Hkv", "d", "page", "topk"))
    G, dev = Hq // Hkv, s["q"].device
    o = torch.empty((B, Nq, Hq, d), dtype=torch.bfloat16, device=dev)
    lse = torch.empty((B, Hq, Nq), dtype=torch.float32, device=dev)
    kp, vp = (s[x].view(-1, BLOCK, Hkv, d) for x in ("kp", "vp"))
    h = torch.arange(Hkv, device=dev)[:, None]
    step = max(1, (1 << 28) // (Hkv * topk * BLOCK * d))
    for b in range(B):
        for i in range(0, Nq, step):
            blk = s["blocks"][b, i:i + step].long()  # [C, Hkv, topk]
            C = blk.shape[0]
            pos = s["lens"][b].long() - Nq + torch.arange(i, i + C, device=dev)
            at = blk.clamp(min=0)
            at = s["table"][b].long()[at * BLOCK // page] * (page // BLOCK) + at % (page // BLOCK)
            key = blk[..., None] * BLOCK + torch.arange(BLOCK, device=dev)
            seen = ((blk >= 0)[..., None] & (key <= pos[:, None, None, None])).view(C, Hkv, topk * BLOCK)
            k, v = (torch.where(seen[..., None], x[at, :, h].view(C, Hkv, topk * BLOCK, d).float(), 0.0)
                    for x in (kp, vp))
            q = s["q"][b, i:i + C].float().view(C, Hkv, G, d)
            x = (q @ k.transpose(2, 3)).mul_(s["scale"]).masked_fill_(~seen[:, :, None], -math.inf)
            m = x.amax(-1, keepdim=True)
            p = x.sub_(m).exp_()
            l = p.sum(-1, keepdim=True)
            o[b, i:i + C] = (p @ v / l).view(C, Hq, d).to(torch.bfloat16)
            lse[b, :, i:i + C] = (m + l.log()).view(C, Hq).T
    return o, lse


def run(s):
    if not own:
        return {"tables": _plain_tables, "shared": _plain_shared, "bounds": _plain_bounds, "select": _plain_select,
                "attend": _plain_attend}[s["op"]](s)
    from exact_io_aware_14_gb300 import _native as A
    if s["op"] == "tables":
        count = A.kvcache_release_paged(s["table"], s["lens"], s["keep"], s["free"], s["count"], s["page"])
        granted, slots, count = A.kvcache_reserve_paged(s["table"], s["keep"], s["new"], s["free"], count, s["page"],
                                                        s["Nn"])
        return s["table"], s["free"], granted, slots, count
    if s["op"] == "shared":
        return A.decode_paged_shared(s["q"], s["kp"], s["vp"], s["table"], s["lens"], s["shared"], s["scale"])
    if s["op"] == "bounds":
        A.kvcache_bounds_paged(s["kp"], s["kb"], s["table"], s["lens"], s["Nn"], new_lens=s["new"])
        return s["kb"]
    if s["op"] == "select":
        return A.select_blocks_paged(s["q"], s["kb"], s["table"], s["lens"], s["topk"], sink=1, local=1)
    return A.attend_blocks_paged(s["q"], s["kp"], s["vp"], s["table"], s["lens"], s["blocks"], s["scale"])


# --------------------------------------------------------------------------- work
def work(case):
    """Inputs once, outputs once: bytes; multiplications and additions of the products: flops.  Lengths at their mean."""
    c = case
    B, page = c["B"], c["page"]
    if c["op"] == "tables":
        tokens = 0.9 * B * ((c["Nn"] + 1) // 2 + c["Nn"]) / 2
        back = 0.1 * B * (c["hi"] / 2 / page + 0.5)
        return {"bytes": 20 * B + 8 * B * c["Nn"] + 8 * (tokens / page + back), "flops": 0}
    Hkv, d = c["Hkv"], c["d"]
    if c["op"] == "bounds":
        tokens = B * ((c["Nn"] + 1) // 2 + c["Nn"]) / 2
        return {"bytes": (tokens + tokens / BLOCK * 2) * Hkv * d * 2, "flops": 2 * tokens * Hkv * d}
    Nq, Hq = c["Nq"], c["Hq"]
    mean = max((c["lo"] + c["hi"]) / 2, Nq)
    if c["op"] == "shared":
        return {"bytes": (c["shared"] + B * mean) * Hkv * d * 4 + B * Nq * Hq * (d * 4 + 4),
                "flops": 4 * d * Hq * Nq * B * (c["shared"] + mean)}
    blocks = mean / BLOCK
    if c["op"] == "select":
        return {"bytes": B * blocks * Hkv * d * 4 + B * Nq * (Hq * d * 2 + Hkv * c["topk"] * 4),
                "flops": 4 * d * B * Nq * Hq * blocks}
    listed_ = min(c["topk"], blocks)
    return {"bytes": B * min(Nq * listed_, blocks) * BLOCK * Hkv * d * 4
            + B * Nq * (Hq * (d * 4 + 4) + Hkv * c["topk"] * 4),
            "flops": 4 * d * B * Nq * Hq * listed_ * BLOCK}


# --------------------------------------------------------------------------- from the definition, in 64 bits
def _exact_tables(c):
    """One page at a time, as a host would keep its lists."""
    page = c["page"]
    table, free = c["table"].tolist(), c["free"].tolist()
    lens, keep, new, top = c["lens"].tolist(), c["keep"].tolist(), c["new"].tolist(), int(c["count"])
    for b in reversed(range(c["B"])):
        for blk in reversed(range(-(-keep[b] // page), -(-lens[b] // page))):
            free[top] = table[b][blk]
            top += 1
    granted, wanted = [], 0
    slots = torch.full((c["B"], c["Nn"]), -1, dtype=torch.int64)
    have = top
    for b in range(c["B"]):
        first, end = -(-keep[b] // page), -(-(keep[b] + new[b]) // page)
        wanted += end - first
        if wanted > have and end > first:
            granted.append(0)
            continue
        for blk in range(first, end):
            top -= 1
            table[b][blk] = free[top]
        granted.append(new[b])
        at = torch.arange(keep[b], keep[b] + new[b])
        slots[b, :new[b]] = torch.tensor(table[b])[at // page] * page + at % page
    dev = c["table"].device
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)
    return [i32(table), i32(free), i32(granted), slots.to(dev), i32([top])]


def _exact_attention(c, keys_of):
    """Softmax attention of each query row over the keys that keys_of(b, i, h) gives: (k, v) [n, d]."""
    B, Nq, Hq, Hkv, d = (c[n] for n in ("B", "Nq", "Hq", "Hkv", "d"))
    G = Hq // Hkv
    o = torch.zeros((B, Nq, Hq, d), dtype=torch.float64, device=c["q"].device)
    lse = torch.full((B, Hq, Nq), -math.inf, dtype=torch.float64, device=c["q"].device)
    for b in range(B):
        for i in range(Nq):
            for h in range(Hkv):
                k, v = keys_of(b, i, h)
                x = c["scale"] * (c["q"][b, i, h * G:(h + 1) * G].double() @ k.T)
                lse[b, h * G:(h + 1) * G, i] = torch.logsumexp(x, -1)
                o[b, i, h * G:(h + 1) * G] = torch.softmax(x, -1) @ v
    return [o, lse]


def exact(case, seed):
    c = prepare(case, seed)
    B, page = c["B"], c["page"]
    if c["op"] == "tables":
        return _exact_tables(c)
    lens, dev = c["lens"].tolist(), c["lens"].device
    if c["op"] == "bounds":
        kb, new = c["kb"].double(), c["new"].tolist()
        for b in range(B):
            for blk in range((lens[b] - new[b]) // BLOCK, (lens[b] - 1) // BLOCK + 1):
                pg, row = int(c["table"][b, blk * BLOCK // page]), blk * BLOCK % page
                x = c["kp"][pg, row:row + min(BLOCK, lens[b] - blk * BLOCK)].double()
                kb[pg, row // BLOCK, :, 0], kb[pg, row // BLOCK, :, 1] = x.min(0).values, x.max(0).values
        return kb
    Nq, Hq, Hkv, d = c["Nq"], c["Hq"], c["Hkv"], c["d"]
    G = Hq // Hkv
    if c["op"] == "select":
        topk = c["topk"]
        out = torch.full((B, Nq, Hkv, topk), -1, dtype=torch.int32, device=dev)
        for b in range(B):
            nb = (lens[b] - 1) // BLOCK + 1
            kb = c["kb"][c["table"][b, :-(-lens[b] // page)].long()].view(-1, Hkv, 2, d)[:nb].double()
            last = (lens[b] - Nq + torch.arange(Nq, device=dev)) // BLOCK
            j = torch.arange(nb, device=dev)
            for h in range(Hkv):
                step = max(1, (1 << 27) // (nb * max(d, nb)))
                for i in range(0, Nq, step):
                    x = None  # the largest over the group's heads of the sum of max(q lo, q hi)
                    for g in range(G):
                        q = c["q"][b, i:i + step, h * G + g].double()[:, None]
                        y = torch.maximum(q * kb[:, h, 0], q * kb[:, h, 1]).sum(-1)
                        x = y if x is None else torch.maximum(x, y)
                    end = last[i:i + step, None]
                    x = torch.where((j == 0) | (j == end), math.inf, x)
                    ahead = (x[:, None, :] > x[:, :, None]) | ((x[:, None, :] == x[:, :, None]) & (j < j[:, None]))
                    rank = (ahead & (j <= end[:, :, None])).sum(-1)
                    chosen = (rank < topk) & (j <= end)
                    place = chosen.cumsum(-1) - 1
                    r, col = chosen.nonzero(as_tuple=True)
                    out[b, i + r, h, place[r, col]] = col.to(torch.int32)
        return out
    if B * Nq * Hkv > 20000:
        return None  # a row at a time takes too long
    if c["op"] == "shared":
        rows = {}

        def keys_of(b, i, h):
            if (b, h) not in rows:
                rows.clear()
                pg = c["table"][b, :-(-lens[b] // page)].long()
                rows[b, h] = [c[x][pg, :, h].double().reshape(-1, d)[:lens[b]] for x in ("kp", "vp")]
            n = lens[b] - Nq + 1 + i
            return [x[:n] for x in rows[b, h]]
    else:
        blocks = c["blocks"].tolist()

        def keys_of(b, i, h):
            at = torch.cat([torch.arange(j * BLOCK, min((j + 1) * BLOCK, lens[b] - Nq + 1 + i))
                            for j in blocks[b][i][h] if j >= 0]).to(dev)
            pg, row = c["table"][b].long()[at // page], at % page
            return [c[x][pg, row, h].double() for x in ("kp", "vp")]
    return _exact_attention(c, keys_of)

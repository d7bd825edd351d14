"""Plain forms, in 64 bits or on the host, of the operators on a paged cache,
and the error bounds that the tests hold the kernels to (the roundings are
counted as in _serving.py)."""
import torch

BLOCK = 64


def pools(g, num_pages, page, Hkv, d, n=2):
    return [torch.randn((num_pages, page, Hkv, d), generator=g).to(torch.bfloat16) for _ in range(n)]


def tables(g, B, blocks, shared_blocks, spare=2):
    """(block_table, num_pages): a random page for each block, the first shared_blocks in common."""
    num = shared_blocks + B * (blocks - shared_blocks) + spare
    perm = torch.randperm(num, generator=g).to(torch.int32)
    own = perm[shared_blocks:num - spare].view(B, blocks - shared_blocks)
    return torch.cat((perm[:shared_blocks].expand(B, shared_blocks), own), 1).contiguous(), num


def rows_of(pool, table, page, b, h, keys):
    keys = torch.as_tensor(keys)
    return pool[table[b].long()[keys // page], keys % page, h].double()


def attend(q, kp, vp, table, page, scale, keys_of):
    """Attention of each row over the keys that keys_of(b, i, hkv) lists, in 64 bits.  Returns o, lse and the bounds on
    their errors before o's rounding to bf16:
      scores: fp32 sums of d products in any order, truncated at worst (2^-23 an addition), and the product with the
      scale rounded: ds;
      weights: rounded to bf16 (2^-8 of each), shifted by the scores' error (2 ds): on sum p |v|;
      2^-19 of the largest value for what the rest rounds (sums, the joining of splits)."""
    B, Nq, Hq, d = q.shape
    G = Hq // kp.shape[2]
    o = torch.zeros((B, Nq, Hq, d), dtype=torch.float64)
    lse = torch.full((B, Hq, Nq), -float("inf"), dtype=torch.float64)
    eo, el = torch.zeros_like(o), torch.zeros_like(lse)
    for b in range(B):
        for i in range(Nq):
            for h in range(Hq // G):
                keys = keys_of(b, i, h)
                if len(keys) == 0:
                    continue
                kk, vv = (rows_of(x, table, page, b, h, keys) for x in (kp, vp))
                hs = slice(h * G, (h + 1) * G)
                qq = q[b, i, hs].double()
                s = scale * (qq @ kk.T)
                p = torch.softmax(s, -1)
                o[b, i, hs], lse[b, hs, i] = p @ vv, torch.logsumexp(s, -1)
                ds = 2.0 ** -23 * d * abs(scale) * (qq.abs() @ kk.abs().T).amax(-1, keepdim=True) + 2.0 ** -22 * s.abs().amax(-1, keepdim=True)
                eo[b, i, hs] = (2.0 ** -8 + 2 * ds) * (p @ vv.abs()) + 2.0 ** -19 * vv.abs().max()
                el[b, hs, i] = ds[:, 0] + 2.0 ** -20 * (1 + lse[b, hs, i].abs())
    return o, lse, eo, el


def check(o, lse, want, what=""):
    """o (bf16) and lse against attend's results: o is rounded by half a step, 2^-8 of it."""
    wo, wl, eo, el = want
    o, lse = o.double().cpu(), lse.double().cpu()
    bad = ~((o - wo).abs() <= eo + 2.0 ** -8 * (wo.abs() + eo))
    assert not bad.any(), "%s: %d of %d outputs outside their bound, the first at %s: %g, want %g +- %g" % (
        what, int(bad.sum()), bad.numel(), tuple(bad.nonzero()[0].tolist()), o[bad][0], wo[bad][0], eo[bad][0])
    empty = wl == -float("inf")
    assert torch.equal(lse == -float("inf"), empty), what
    bad = ~((lse - wl).abs() <= el) & ~empty
    assert not bad.any(), "%s: %d log-sum-exps outside their bound: %s, want %s" % (
        what, int(bad.sum()), lse[bad][:4].tolist(), wl[bad][:4].tolist())


def reserve(table, seqlens, new_lens, free, count, page, max_new):
    """(table, granted, slots, count) one page at a time; lists."""
    table = [list(r) for r in table]
    granted, slots, top, wanted = [], [], count, 0
    for b, (n, m) in enumerate(zip(seqlens, new_lens)):
        first, end = -(-n // page), -(-(n + m) // page)
        wanted += end - first
        if end > first and wanted > count:
            granted.append(0)
            slots.append([-1] * max_new)
            continue
        for blk in range(first, end):
            top -= 1
            table[b][blk] = free[top]
        granted.append(m)
        slots.append([table[b][(n + i) // page] * page + (n + i) % page for i in range(m)] + [-1] * (max_new - m))
    return table, granted, slots, top


def release(table, seqlens, keep, free, count, page):
    free = list(free)
    for b in reversed(range(len(seqlens))):
        for blk in reversed(range(-(-keep[b] // page), -(-seqlens[b] // page))):
            free[count] = table[b][blk]
            count += 1
    return free, count


def bounds(kp, table, page, seqlens, new_lens, kb):
    """kb with the bounds of the blocks that the last new_lens tokens reach."""
    kb = kb.clone()
    for b, (L, n) in enumerate(zip(seqlens, new_lens)):
        for blk in range((L - n) // BLOCK, (L + BLOCK - 1) // BLOCK) if n else ():
            pg, row = int(table[b, blk * BLOCK // page]), blk * BLOCK % page
            x = kp[pg, row:row + min(BLOCK, L - blk * BLOCK)]
            kb[pg, row // BLOCK] = torch.stack((x.amin(0), x.amax(0)), 1)
    return kb


def scores(q, lo, hi):
    """[G, d] x [n, d] -> [n], in 64 bits; NaN ranks as +inf."""
    q, lo, hi = q.double()[:, None], lo.double(), hi.double()
    s = (q.clamp(min=0) * hi + q.clamp(max=0) * lo).sum(-1)
    return torch.where(s.isnan(), float("inf"), s).amax(0)


def select(q, kb, table, page, seqlens, topk, sink, local):
    B, Nq, Hq, d = q.shape
    Hkv = kb.shape[2]
    G = Hq // Hkv
    out = torch.full((B, Nq, Hkv, topk), -1, dtype=torch.int32)
    for b in range(B):
        flat = kb[table[b].long()].reshape(-1, Hkv, 2, d)
        for i in range(Nq):
            pos = seqlens[b] - Nq + i
            nb = pos // BLOCK + 1 if pos >= 0 else 0
            for h in range(Hkv):
                if nb <= topk:
                    chosen = list(range(nb))
                else:
                    s = scores(q[b, i, h * G:(h + 1) * G], flat[:nb, h, 0], flat[:nb, h, 1]).tolist()
                    forced = list(range(sink)) + list(range(nb - local, nb))
                    rest = sorted(range(sink, nb - local), key=lambda j: (-s[j], j))
                    chosen = sorted(forced + rest[:topk - len(forced)])
                out[b, i, h, :len(chosen)] = torch.tensor(chosen, dtype=torch.int32)
    return out

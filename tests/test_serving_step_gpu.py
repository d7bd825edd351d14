"""GPU: the operators together, as a serving loop and a training step use them."""
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


@pytest.mark.parametrize("fp8", [False, True])
def test_prompt_then_tokens(fp8):
    """A padded batch of prompts, then tokens one at a time: norms and rotation, append, decode; the step captured
    once and replayed.  Every step's attention is compared with 64-bit attention over what the cache then holds, and
    the cache with the keys and values that went in."""
    B, Hq, Hkv, d, page, Nn, steps = 3, 8, 2, 128, 64, 150, 5
    g = torch.Generator().manual_seed(90)
    lens = torch.tensor([150, 63, 97], dtype=torch.int32)
    mb = 4
    num_pages = B * mb + 1
    table = torch.randperm(num_pages, generator=g)[:B * mb].view(B, mb).to(torch.int32).cuda()
    dtype = torch.float8_e4m3fn if fp8 else torch.bfloat16
    pools = [torch.full((num_pages, page, Hkv, d), 0xFF, dtype=torch.uint8 if fp8 else torch.int16,
                        device="cuda").view(dtype) for _ in range(2)] if fp8 else [
        torch.full((num_pages, page, Hkv, d), float("nan"), dtype=dtype, device="cuda") for _ in range(2)]
    scales = [torch.zeros((num_pages, Hkv), device="cuda") for _ in range(2)] if fp8 else []
    rope = _native.rope_table(mb * page, d)
    wq, wk = (1 + 0.1 * torch.randn(d, generator=g).cuda() for _ in range(2))
    append = _native.kvcache_append_paged_fp8 if fp8 else _native.kvcache_append_paged

    def step(qkv, seqlens, after, new_lens, pos):
        q, k, v = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:]
        q, k = _native.qk_norm_rope(q, k, wq, wk, 1e-6, rope, pos)
        append(k, v, *pools, *scales, table, seqlens, new_lens=new_lens, seqlens_out=after)
        return q, k, v

    def attend(q, seqlens):
        if fp8:
            return _native.decode_paged_fp8(q, *pools, *scales, table, seqlens, d ** -0.5)
        return _native.decode_paged(q, *pools, table, seqlens, d ** -0.5, chunk=128)

    prompt = torch.randn((B, Nn, Hq + 2 * Hkv, d), generator=g).to(torch.bfloat16).cuda()
    seqlens = torch.zeros(B, dtype=torch.int32, device="cuda")
    after = torch.empty_like(seqlens)
    _, k, v = step(prompt, seqlens, after, lens.cuda(), None)
    assert after.tolist() == lens.tolist()
    ks, vs = ([x[b, :int(lens[b])].cpu() for b in range(B)] for x in (k, v))
    # one decode step, captured: its inputs and lengths are updated in place between replays
    token = torch.zeros((B, 1, Hq + 2 * Hkv, d), dtype=torch.bfloat16, device="cuda")
    seqlens.copy_(after)
    pos = seqlens.view(B, 1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q, k, v = step(token, seqlens, after, None, pos)
        o, lse = attend(q, after)
        seqlens.copy_(after)
    for t in range(steps):
        token.copy_(torch.randn(token.shape, generator=g).to(torch.bfloat16))
        graph.replay()
        now = [int(x) for x in after.tolist()]
        assert now == [int(lens[b]) + t + 1 for b in range(B)]
        kc, vc = ([], [])
        n = max(now)
        full = []
        for i, (pool, new, old) in enumerate(zip(pools, (k, v), (ks, vs))):
            val = pool.float().cpu().double()
            if fp8:
                val = val * scales[i].cpu().double()[:, None, :, None]
            rows = S.paged_rows(val, table.cpu(), n)
            for b in range(B):
                old[b] = torch.cat((old[b], new[b].cpu()))
                got, want = rows[b, :now[b]], old[b].double()
                if fp8:   # two roundings at most at the smallest codes: a scale raised after a value was stored
                    sc = S.paged_rows(scales[i].cpu().double()[:, None, :, None].expand(-1, page, -1, 1), table.cpu(),
                                      n)[b, :now[b]]
                    assert ((got - want).abs() <= torch.maximum(2.0 ** -4 * want.abs(), 2.0 ** -9 * sc)).all()
                else:
                    assert torch.equal(got, want)
            full.append(rows)
        o64, lse64, eo, el = S.decode(q.cpu(), *full, now, d ** -0.5)
        S.assert_within(o, o64, eo + 2.0 ** -8 * (o64.abs() + eo), "o at step %d" % t)
        S.assert_within(lse, lse64, el, "lse at step %d" % t)
    assert _native.attn_get_device_status() == 0


def test_training_step():
    """Norms and rotation before the training forward, and their backward pass with the gradients that attention
    gives: compared with 64-bit autograd through the whole step."""
    B, N, Hq, Hkv, d = 2, 70, 4, 2, 64
    g = torch.Generator().manual_seed(91)
    qkv = torch.randn((B, N, Hq + 2 * Hkv, d), generator=g).to(torch.bfloat16)
    wq, wk = (1 + 0.1 * torch.randn(d, generator=g) for _ in range(2))
    rope = _native.rope_table(N, d, device="cpu")
    do = torch.randn((B, N, Hq, d), generator=g).double()
    qc = qkv.cuda()
    q, k, v = qc[:, :, :Hq], qc[:, :, Hq:Hq + Hkv], qc[:, :, Hq + Hkv:]
    r = (rope[0].cuda(), rope[1].cuda())
    qo, ko = _native.qk_norm_rope(q, k, wq.cuda(), wk.cuda(), 1e-6, r)
    o, lse = _native.forward(qo, ko, v.contiguous(), 1, d ** -0.5)
    # 64-bit step
    x = qkv.double().requires_grad_()
    w = [t.double().requires_grad_() for t in (wq, wk)]
    cs = S.angles(rope, torch.arange(N).expand(B, N))
    turned = []
    for part, wt in ((x[:, :, :Hq], w[0]), (x[:, :, Hq:Hq + Hkv], w[1])):
        y = part * (part.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * wt
        a, b = y[..., :d // 2], y[..., d // 2:]
        turned.append(torch.cat((a * cs[0] - b * cs[1], b * cs[0] + a * cs[1]), -1))
    turned[0].retain_grad(), turned[1].retain_grad()
    kk, vv = (t.repeat_interleave(Hq // Hkv, 2) for t in (turned[1], x[:, :, Hq + Hkv:]))
    s = torch.einsum("bihd,bjhd->bhij", turned[0], kk) * d ** -0.5
    s = s.masked_fill(torch.ones(N, N).triu(1).bool(), -float("inf"))
    o64 = torch.einsum("bhij,bjhd->bihd", s.softmax(-1), vv)
    # the workloads' bar for bf16 attention, here with q and k rounded to bf16 before it as well
    assert (o.double().cpu() - o64.detach()).abs().max() <= 4e-2
    (o64 * do).sum().backward()
    gq, gk = (t.grad.to(torch.bfloat16) for t in turned)
    dq, dk, dwq, dwk = _native.qk_norm_rope_bwd(gq.cuda(), gk.cuda(), q, k, wq.cuda(), wk.cuda(), 1e-6, r)
    # the incoming gradients were rounded to bf16: 2^-8 of each, through R^T, w and the norm (a projection)
    for got, part, gy, wt, dw, lo, hi in ((dq, qkv[:, :, :Hq], gq, wq, dwq, 0, Hq),
                                          (dk, qkv[:, :, Hq:Hq + Hkv], gk, wk, dwk, Hq, Hq + Hkv)):
        want = x.grad[:, :, lo:hi]
        rr = (part.double().square().mean(-1, keepdim=True) + 1e-6).rsqrt()
        size = 2.0 ** -8 * rr * float(wt.abs().max()) * gy.double().norm(dim=-1, keepdim=True) * 2
        S.assert_within(got, want, 2.0 ** -8 * (want.abs() + size) + size, "gradient")
        w64 = w[0].grad if lo == 0 else w[1].grad
        xr = part.double() * rr
        terms = (xr.abs() * gy.double().norm(dim=-1, keepdim=True)).reshape(-1, d).sum(0)
        S.assert_within(dw, w64, (2.0 ** -8 + 2.0 ** -16) * terms, "weight gradient")
    assert _native.attn_get_device_status() == 0


def test_positions_written_by_earlier_kernels_of_the_chain():
    """Steps in a row without any other kernel between them, so that each starts while the one before ends: the norms
    take as positions the lengths that the append two launches earlier wrote."""
    B, Hq, Hkv, d, page, steps = 40, 8, 2, 128, 64, 24
    g = torch.Generator().manual_seed(92)
    pools = [torch.zeros((B, page, Hkv, d), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
             for _ in range(2)]
    scales = [torch.zeros((B, Hkv), device="cuda") for _ in range(2)]
    table = torch.arange(B, dtype=torch.int32, device="cuda")[:, None].contiguous()
    rope = _native.rope_table(page, d)
    w = torch.ones(d, device="cuda")
    qkv = torch.randn((B, 1, Hq + 2 * Hkv, d), generator=g).to(torch.bfloat16).cuda()
    parts = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:]
    lens = [torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(2)]

    def chain():
        got = []
        for t in range(steps):
            before, after = lens[t % 2], lens[1 - t % 2]
            q, k = _native.qk_norm_rope(parts[0], parts[1], w, w, 1e-6, rope, before.view(B, 1))
            _native.kvcache_append_paged_fp8(k, parts[2], *pools, *scales, table, before, seqlens_out=after)
            _native.decode_paged_fp8(q, *pools, *scales, table, after, 0.09)
            got.append((q, k))
        return got

    want = [_native.qk_norm_rope(parts[0], parts[1], w, w, 1e-6, rope,
                                 torch.full((B, 1), t, dtype=torch.int32, device="cuda")) for t in range(steps)]
    first = chain()
    lens[0].zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = chain()
    for _ in range(3):
        lens[0].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert lens[0].tolist() == [steps] * B
        for got in (first, again):
            for a, b in zip(got, want):
                assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert _native.attn_get_device_status() == 0


def test_status_is_read_in_one_round_trip():
    """Problems of several kernel units are reported once and cleared together; a call costs a launch and one copy (under
    two copies of a word as measured; six words read one after the other took nine), not a round trip a unit."""
    import time
    x = torch.randn((1, 1, 2, 64), device="cuda").to(torch.bfloat16)
    _native.qk_norm_rope(x, None, None, None, rope=_native.rope_table(4, 64),
                         positions=torch.tensor([[9]], dtype=torch.int32, device="cuda"))
    pools = [torch.zeros((1, 64, 2, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    _native.kvcache_append_paged(x, x, *pools, torch.zeros((1, 1), dtype=torch.int32, device="cuda"),
                                 torch.tensor([64], dtype=torch.int32, device="cuda"))
    assert _native.attn_get_device_status() == _native.ATTN_ERR_DEVICE_ARG
    assert _native.attn_get_device_status() == 0
    word = torch.zeros(1, device="cuda")

    def least(f):
        times = []
        for _ in range(300):
            torch.cuda.synchronize()
            t = time.perf_counter()
            f()
            times.append(time.perf_counter() - t)
        return min(times)

    assert least(_native.attn_get_device_status) < 4 * least(word.item)


def test_prompt_behind_a_prefix_attended_in_blocks():
    """A prompt appended in one call behind keys that are there already, then attended 64 new rows at a time."""
    B, Hq, Hkv, d, page, L, n = 2, 6, 2, 64, 128, 40, 150
    g = torch.Generator().manual_seed(93)
    pools = [torch.full((4, page, Hkv, d), 0x7F, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
             for _ in range(2)]
    scales = [torch.zeros((4, Hkv), device="cuda") for _ in range(2)]
    table = torch.tensor([[2, 0], [3, 1]], dtype=torch.int32, device="cuda")
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    after = torch.empty_like(lens)
    for m in (L, n):
        k, v = (torch.randn((B, m, Hkv, d), generator=g).to(torch.bfloat16).cuda() for _ in range(2))
        _native.kvcache_append_paged_fp8(k, v, *pools, *scales, table, lens, seqlens_out=after)
        lens, after = after, lens
    q = torch.randn((B, n, Hq, d), generator=g).to(torch.bfloat16)
    parts = []
    for i in range(0, n, 64):
        m = min(64, n - i)
        parts.append(_native.decode_paged_fp8(q[:, i:i + m].contiguous().cuda(), *pools, *scales, table,
                                              torch.full((B,), L + i + m, dtype=torch.int32, device="cuda"), 0.125))
    assert _native.attn_get_device_status() == 0
    k, v = (S.paged_rows(p.float().cpu().double() * s.cpu().double()[:, None, :, None], table.cpu(), L + n)
            for p, s in zip(pools, scales))
    o, lse, eo, el = S.decode(q, k, v, [L + n] * B, 0.125)
    S.assert_within(torch.cat([p[0] for p in parts], 1), o, eo + 2.0 ** -8 * (o.abs() + eo), "o")
    S.assert_within(torch.cat([p[1] for p in parts], 2), lse, el, "lse")

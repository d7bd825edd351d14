"""GPU: norms and rotation of queries and keys, forward and backward, against
the formulas in 64 bits."""
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


def _inputs(B, N, Hq, Hkv, d, rot, seed, positions=True, extra=0, max_pos=600):
    """q, k as parts of a projection with `extra` more heads a token (0: dense tensors), weights, tables, positions."""
    g = torch.Generator().manual_seed(seed)
    if extra:
        x = torch.randn((B, N, Hq + Hkv + extra, d), generator=g).to(torch.bfloat16)
        q, k = x[:, :, :Hq], x[:, :, Hq:Hq + Hkv]
        xc = x.cuda()
        qc, kc = xc[:, :, :Hq], xc[:, :, Hq:Hq + Hkv]
    else:
        q, k = (torch.randn((B, N, H, d), generator=g).to(torch.bfloat16) for H in (Hq, Hkv))
        qc, kc = q.cuda(), k.cuda()
    wq, wk = (1 + 0.3 * torch.randn(d, generator=g) for _ in range(2))
    rope = _native.rope_table(max_pos, rot, device="cpu") if rot else None
    pos = torch.randint(0, max_pos, (B, N), generator=g, dtype=torch.int32) if positions else None
    at = pos if positions else torch.arange(N).expand(B, N)
    return g, q, k, qc, kc, wq, wk, rope, pos, S.angles(rope, at)


def _gpu(rope):
    return None if rope is None else (rope[0].cuda(), rope[1].cuda())


SHAPES = [
    # B, N, Hq, Hkv, d, rot, inter, positions, extra
    (1, 1, 1, 1, 64, 64, False, True, 0),
    (1, 1, 32, 8, 128, 128, False, True, 8),
    (64, 1, 32, 8, 128, 128, False, True, 8),
    (3, 37, 9, 3, 64, 32, True, True, 3),
    (2, 65, 5, 1, 128, 48, False, True, 1),
    (2, 33, 7, 2, 128, 16, True, False, 2),
    (2, 130, 4, 4, 64, 0, False, False, 0),
    (1, 515, 6, 2, 128, 128, True, False, 0),
    (2, 19, 3, 5, 64, 64, False, True, 4),     # more k heads than q heads
]


@pytest.mark.parametrize("B,N,Hq,Hkv,d,rot,inter,positions,extra", SHAPES)
@pytest.mark.parametrize("norm", [True, False])
def test_forward(B, N, Hq, Hkv, d, rot, inter, positions, extra, norm):
    _, q, k, qc, kc, wq, wk, rope, pos, cs = _inputs(B, N, Hq, Hkv, d, rot, 100 + N + d, positions, extra)
    w = (wq.cuda(), wk.cuda()) if norm else (None, None)
    qo, ko = _native.qk_norm_rope(qc, kc, *w, 1e-6, _gpu(rope), None if pos is None else pos.cuda(), inter)
    assert _native.attn_get_device_status() == 0
    for x, wx, got, what in ((q, wq, qo, "q"), (k, wk, ko, "k")):
        y, size = S.norm_rope(x, wx if norm else None, 1e-6, cs, inter)
        # one rounding to bf16, under 16 fp32 roundings of values up to the row's largest
        S.assert_within(got, y, 2.0 ** -8 * y.abs() + 2.0 ** -20 * size, what)


@pytest.mark.parametrize("B,N,Hq,Hkv,d,rot,inter,positions,extra", SHAPES)
@pytest.mark.parametrize("norm", [True, False])
def test_backward(B, N, Hq, Hkv, d, rot, inter, positions, extra, norm):
    g, q, k, qc, kc, wq, wk, rope, pos, cs = _inputs(B, N, Hq, Hkv, d, rot, 200 + N + d, positions, extra)
    gq, gk = (torch.randn((B, N, H, d), generator=g).to(torch.bfloat16) for H in (Hq, Hkv))
    w = (wq.cuda(), wk.cuda()) if norm else (None, None)
    xs = (qc, kc) if norm else (None, None)
    got = _native.qk_norm_rope_bwd(gq.cuda(), gk.cuda(), *xs, *w, 1e-6, _gpu(rope),
                                   None if pos is None else pos.cuda(), inter)
    assert _native.attn_get_device_status() == 0
    for x, wx, dy, dx_got, dw_got, what in ((q, wq, gq, got[0], got[2], "q"), (k, wk, gk, got[1], got[3], "k")):
        dx, err, dw, size = S.norm_rope_bwd(dy, x, wx if norm else None, 1e-6, cs, inter)
        S.assert_within(dx_got, dx, 2.0 ** -8 * dx.abs() + err, "d" + what)
        if norm:
            # at these sizes under 256 fp32 additions lie between a term and the sum
            S.assert_within(dw_got, dw, 2.0 ** -16 * size, "dw" + what)
        else:
            assert dw_got is None


def test_backward_against_differences():
    """dx and dw of the kernel against central differences of the forward formula in 64 bits, along one direction."""
    B, N, H, d, rot = 2, 3, 2, 64, 32
    g, q, k, qc, kc, wq, wk, rope, pos, cs = _inputs(B, N, H, H, d, rot, 5)
    gq, gk = (torch.randn((B, N, H, d), generator=g).to(torch.bfloat16) for _ in range(2))
    dq, _, dwq, _ = _native.qk_norm_rope_bwd(gq.cuda(), gk.cuda(), qc, kc, wq.cuda(), wk.cuda(), 1e-6, _gpu(rope),
                                             pos.cuda())
    v = torch.randn((B, N, H, d), generator=g, dtype=torch.float64)
    vw = torch.randn(d, generator=g, dtype=torch.float64)
    f = lambda x, w: float((S.norm_rope(x, w, 1e-6, cs, False)[0] * gq.double()).sum())
    h = 1e-5
    x, w = q.double(), wq.double()
    num = (f(x + h * v, w) - f(x - h * v, w)) / (2 * h)
    dq = dq.double().cpu()
    assert abs(num - float((dq * v).sum())) <= float((2.0 ** -8 * dq.abs() * v.abs()).sum()) + 1e-4
    num = (f(x, w + h * vw) - f(x, w - h * vw)) / (2 * h)
    dwq = dwq.double().cpu()
    terms = (gq.double().abs().sum() * 8)  # |xr| <= 8 = sqrt(d)
    assert abs(num - float((dwq * vw).sum())) <= 2.0 ** -20 * float(terms) * float(vw.abs().max()) + 1e-4


def test_large_and_repeatable():
    """More rows than the backward pass has threads (every thread walks several): bounds, and the same bits twice."""
    B, N, Hq, Hkv, d = 2, 2500, 16, 4, 128
    g, q, k, qc, kc, wq, wk, rope, pos, cs = _inputs(B, N, Hq, Hkv, d, 128, 9, True, 4, 4000)
    gq, gk = (torch.randn((B, N, H, d), generator=g).to(torch.bfloat16) for H in (Hq, Hkv))
    args = (gq.cuda(), gk.cuda(), qc, kc, wq.cuda(), wk.cuda(), 1e-6, _gpu(rope), pos.cuda())
    a, b = _native.qk_norm_rope_bwd(*args), _native.qk_norm_rope_bwd(*args)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    dx, err, dw, size = S.norm_rope_bwd(gq, q, wq, 1e-6, cs, False)
    S.assert_within(a[0], dx, 2.0 ** -8 * dx.abs() + err, "dq")
    S.assert_within(a[2], dw, 2.0 ** -16 * size, "dwq")
    dx, err, dw, size = S.norm_rope_bwd(gk, k, wk, 1e-6, cs, False)
    S.assert_within(a[1], dx, 2.0 ** -8 * dx.abs() + err, "dk")
    S.assert_within(a[3], dw, 2.0 ** -16 * size, "dwk")


def test_in_place_q_alone_and_empty():
    _, q, k, qc, kc, wq, wk, rope, pos, cs = _inputs(2, 9, 4, 2, 128, 128, 11)
    r = _gpu(rope)
    want = _native.qk_norm_rope(qc, kc, wq.cuda(), wk.cuda(), 1e-6, r, pos.cuda())
    a, b = qc.clone(), kc.clone()
    _native.qk_norm_rope(a, b, wq.cuda(), wk.cuda(), 1e-6, r, pos.cuda(), out=(a, b))
    assert torch.equal(a, want[0]) and torch.equal(b, want[1])
    alone, none = _native.qk_norm_rope(qc, None, wq.cuda(), None, 1e-6, r, pos.cuda())
    assert none is None and torch.equal(alone, want[0])
    only_k = _native.qk_norm_rope(qc, kc, None, wk.cuda(), 1e-6, r, pos.cuda())
    assert torch.equal(only_k[1], want[1])
    e = torch.empty((2, 0, 4, 128), dtype=torch.bfloat16, device="cuda")
    assert _native.qk_norm_rope(e, e, None, None)[0].shape == e.shape
    w = torch.ones(128, device="cuda")
    g = _native.qk_norm_rope_bwd(e, e, e, e, w, w)
    assert g[2].abs().max() == 0 and g[3].abs().max() == 0
    assert _native.attn_get_device_status() == 0


def test_in_place_long_and_odd_heads():
    """Sizes that take the long form, in place, with head counts that four do not divide and that they do."""
    for Hq, Hkv in ((9, 3), (16, 4)):
        _, q, k, qc, kc, wq, wk, rope, pos, cs = _inputs(2, 1500, Hq, Hkv, 128, 128, 12, True, 0, 4000)
        r = _gpu(rope)
        want = _native.qk_norm_rope(qc, kc, wq.cuda(), wk.cuda(), 1e-6, r, pos.cuda())
        _native.qk_norm_rope(qc, kc, wq.cuda(), wk.cuda(), 1e-6, r, pos.cuda(), out=(qc, kc))
        assert torch.equal(qc, want[0]) and torch.equal(kc, want[1])
        for x, wx, got in ((q, wq, want[0]), (k, wk, want[1])):
            y, size = S.norm_rope(x, wx, 1e-6, cs, False)
            S.assert_within(got, y, 2.0 ** -8 * y.abs() + 2.0 ** -20 * size, "rows")


def test_one_norm_only_and_gradients_in_place():
    """A norm on k alone (q rotated only), and the C call's gradients written over the incoming ones."""
    B, N, Hq, Hkv, d = 2, 50, 6, 2, 128
    g, q, k, qc, kc, wq, wk, rope, pos, cs = _inputs(B, N, Hq, Hkv, d, 64, 13)
    r, p = _gpu(rope), pos.cuda()
    gq, gk = (torch.randn((B, N, H, d), generator=g).to(torch.bfloat16) for H in (Hq, Hkv))
    dq, dk, dwq, dwk = _native.qk_norm_rope_bwd(gq.cuda(), gk.cuda(), None, kc, None, wk.cuda(), 1e-6, r, p)
    assert dwq is None
    dx, err, _, _ = S.norm_rope_bwd(gq, q, None, 1e-6, cs, False)
    S.assert_within(dq, dx, 2.0 ** -8 * dx.abs() + err, "dq")
    dx, err, dw, size = S.norm_rope_bwd(gk, k, wk, 1e-6, cs, False)
    S.assert_within(dk, dx, 2.0 ** -8 * dx.abs() + err, "dk")
    S.assert_within(dwk, dw, 2.0 ** -16 * size, "dwk")
    full = _native.qk_norm_rope_bwd(gq.cuda(), gk.cuda(), qc, kc, wq.cuda(), wk.cuda(), 1e-6, r, p)
    a, b = gq.cuda(), gk.cuda()
    dw = [torch.empty(d, device="cuda") for _ in range(2)]
    n = _native.attn_qk_norm_rope_bwd_workspace_size(B, N, Hq, Hkv, d)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    w = [t.cuda() for t in (wq, wk)]
    st = torch.cuda.current_stream().cuda_stream
    rc = _native.lib().attn_qk_norm_rope_bwd(
        a.data_ptr(), b.data_ptr(), qc.data_ptr(), Hq * d, kc.data_ptr(), Hkv * d, w[0].data_ptr(), w[1].data_ptr(),
        1e-6, r[0].data_ptr(), r[1].data_ptr(), r[0].shape[0], 64, 0, p.data_ptr(), a.data_ptr(), b.data_ptr(),
        dw[0].data_ptr(), dw[1].data_ptr(), B, N, Hq, Hkv, d, ws.data_ptr(), n, st)
    assert rc == 0
    for got, want in zip((a, b, *dw), full):
        assert torch.equal(got, want)


# past 2^21 values, where the forward pass takes the long form: four heads an item and one, each rotation
LONG = [
    # B, N, Hq, Hkv, d, rot, inter, positions, extra
    (2, 900, 16, 4, 64, 64, False, True, 3),
    (3, 1100, 9, 3, 64, 32, True, False, 2),
    (2, 850, 16, 8, 64, 64, True, False, 0),
    (2, 1400, 9, 3, 64, 48, False, False, 1),
    (2, 450, 16, 4, 128, 128, True, False, 0),
    (2, 850, 9, 1, 128, 48, True, True, 1),
    (2, 900, 5, 5, 128, 32, False, False, 2),
    (1, 1100, 20, 4, 128, 0, False, False, 0),
    (1, 1701, 12, 0, 128, 96, False, True, 4),        # q alone
]


@pytest.mark.parametrize("B,N,Hq,Hkv,d,rot,inter,positions,extra", LONG)
@pytest.mark.parametrize("norms", ["both", "none", "q", "k"])
def test_long_form(B, N, Hq, Hkv, d, rot, inter, positions, extra, norms):
    """Forward and backward at sizes of the long form, with and without each norm."""
    g, q, k, qc, kc, wq, wk, rope, pos, cs = _inputs(B, N, Hq, Hkv, d, rot, 400 + N + d, positions, extra, 2000)
    gq, gk = (torch.randn((B, N, H, d), generator=g).to(torch.bfloat16) for H in (Hq, Hkv))
    w = [wq if norms in ("both", "q") else None, wk if norms in ("both", "k") and Hkv else None]
    wc = [None if t is None else t.cuda() for t in w]
    r, p = _gpu(rope), None if pos is None else pos.cuda()
    out = _native.qk_norm_rope(qc, kc if Hkv else None, *wc, 1e-6, r, p, inter)
    back = _native.qk_norm_rope_bwd(gq.cuda(), gk.cuda() if Hkv else None, qc, kc if Hkv else None, *wc, 1e-6, r, p,
                                    inter)
    assert _native.attn_get_device_status() == 0
    for i, (x, dy) in enumerate(((q, gq), (k, gk))[:2 if Hkv else 1]):
        y, size = S.norm_rope(x, w[i], 1e-6, cs, inter)
        S.assert_within(out[i], y, 2.0 ** -8 * y.abs() + 2.0 ** -20 * size, "y %d" % i)
        dx, err, dw, size = S.norm_rope_bwd(dy, x, w[i], 1e-6, cs, inter)
        S.assert_within(back[i], dx, 2.0 ** -8 * dx.abs() + err, "dx %d" % i)
        if w[i] is not None:
            S.assert_within(back[2 + i], dw, 2.0 ** -16 * size, "dw %d" % i)


@pytest.mark.parametrize("Hq,Hkv,d,inter", [(24, 8, 128, False), (24, 8, 128, True), (27, 5, 128, False),
                                            (27, 5, 128, True), (24, 8, 64, False), (24, 8, 64, True),
                                            (27, 5, 64, False), (27, 5, 64, True), (53, 11, 64, False)])
def test_past_the_second_level_cache(Hq, Hkv, d, inter):
    """Tensors of more than 129 MB together, whose loads and stores are streamed: every row against 64 bits (formed on the
    GPU, some tokens at a time), dw over all of them."""
    B, N, rot = 4, 2101 * 128 // d, d if Hq % 2 == 0 else d // 2
    positions = Hq % 4 == 0
    gen = torch.Generator(device="cuda").manual_seed(40 + Hq + d)
    x = torch.randn((B, N, Hq + Hkv + 1, d), generator=gen, device="cuda").to(torch.bfloat16)
    xs = x[:, :, :Hq], x[:, :, Hq:Hq + Hkv]
    gs = [torch.randn((B, N, H, d), generator=gen, device="cuda").to(torch.bfloat16) for H in (Hq, Hkv)]
    ws = [1 + 0.3 * torch.randn(d, generator=gen, device="cuda") for _ in range(2)]
    rope = _native.rope_table(N, rot)
    pos = torch.randint(0, N, (B, N), generator=gen, device="cuda", dtype=torch.int32) if positions else None
    at = pos if positions else torch.arange(N, device="cuda").expand(B, N)
    out = _native.qk_norm_rope(*xs, *ws, 1e-6, rope, pos, inter)
    back = _native.qk_norm_rope_bwd(*gs, *xs, *ws, 1e-6, rope, pos, inter)
    assert _native.attn_get_device_status() == 0

    def close(got, want, bound, what):
        bad = (got.double() - want).abs() > bound
        assert not bad.any(), "%s: %d values outside their bound" % (what, int(bad.sum()))

    for i in range(2):
        sums = [0.0, 0.0]
        for n in range(0, N, 300):
            part = slice(n, n + 300)
            cs = S.angles(rope, at[:, part])
            y, size = S.norm_rope(xs[i][:, part], ws[i], 1e-6, cs, inter)
            close(out[i][:, part], y, 2.0 ** -8 * y.abs() + 2.0 ** -20 * size, "y %d" % i)
            dx, err, dw, size = S.norm_rope_bwd(gs[i][:, part], xs[i][:, part], ws[i], 1e-6, cs, inter)
            close(back[i][:, part], dx, 2.0 ** -8 * dx.abs() + err, "dx %d" % i)
            sums = [sums[0] + dw, sums[1] + size]
        # under 256 fp32 additions between a term and the sum here too (under 60 rows a thread, 304 blocks)
        close(back[2 + i], sums[0], 2.0 ** -16 * sums[1], "dw %d" % i)


@pytest.mark.parametrize("B,N,Hq,Hkv,d,rot,inter,positions,extra", SHAPES)
@pytest.mark.parametrize("which", ["q", "w", "all", "plain"])
def test_gradients_through_autograd(B, N, Hq, Hkv, d, rot, inter, positions, extra, which):
    """Outputs of inputs that require gradients carry a graph; its gradients are qk_norm_rope_bwd's, against the formula
    in 64 bits: of the inputs alone, the weights alone, both, and of a rotation without norms."""
    g, q, k, qc, kc, wq, wk, rope, pos, cs = _inputs(B, N, Hq, Hkv, d, rot, 300 + N + d, positions, extra)
    gq, gk = (torch.randn((B, N, H, d), generator=g).to(torch.bfloat16) for H in (Hq, Hkv))
    x = [qc.detach(), kc.detach()]
    w = [None, None] if which == "plain" else [wq.cuda(), wk.cuda()]
    leaves = (x[:1] if which == "q" else x if which == "plain" else w if which == "w" else x + w)
    for t in leaves:
        t.requires_grad_()
    p = None if pos is None else pos.cuda()
    outs = _native.qk_norm_rope(*x, *w, 1e-6, _gpu(rope), p, inter)
    assert all(o.requires_grad for o in outs)
    with torch.no_grad():
        plain = _native.qk_norm_rope(*x, *w, 1e-6, _gpu(rope), p, inter)
    assert not any(o.requires_grad for o in plain) and all(torch.equal(a, b) for a, b in zip(outs, plain))
    (outs[0].float() * gq.cuda().float()).sum().backward(retain_graph=True)    # one output's part alone
    outs[1].backward(gk.cuda())                                               # and the other's added to it
    for i, (t, wt, xc, wx, dy) in enumerate(((x[0], w[0], q, wq, gq), (x[1], w[1], k, wk, gk))):
        dx, err, dw, size = S.norm_rope_bwd(dy, xc, None if which == "plain" else wx, 1e-6, cs, inter)
        if t.requires_grad:
            S.assert_within(t.grad, dx, 2.0 ** -8 * dx.abs() + err, "dx %d" % i)
        else:
            assert t.grad is None
        if wt is not None and wt.requires_grad:
            S.assert_within(wt.grad, dw, 2.0 ** -16 * size, "dw %d" % i)
    assert _native.attn_get_device_status() == 0


def test_autograd_edges():
    """Gradients that are expanded, strided or off a 16-byte boundary, k left out or without heads, out=, a captured
    step, and an input changed between the passes."""
    d = 64
    g = torch.Generator().manual_seed(31)
    base = torch.randn((2, 5, 3, d), generator=g).to(torch.bfloat16).cuda()
    w0 = (1 + 0.3 * torch.randn(d, generator=g)).cuda()
    dy = torch.randn((2, 5, 3, d), generator=g).to(torch.bfloat16).cuda()

    def grads(dy, k=None, kw=None):
        q, w = base.clone().requires_grad_(), w0.clone().requires_grad_()
        o, _ = _native.qk_norm_rope(q, k, w, kw)
        return torch.autograd.grad(o, (q, w), dy)

    want = _native.qk_norm_rope_bwd(dy, None, base, None, w0, None)
    odd = torch.empty(dy.numel() + 1, dtype=torch.bfloat16, device="cuda")[1:].view_as(dy).copy_(dy)
    wide = torch.empty((2, 5, 3, 2 * d), dtype=torch.bfloat16, device="cuda")[..., :d].copy_(dy)
    none = torch.empty((2, 5, 0, d), dtype=torch.bfloat16, device="cuda")
    for got in (grads(dy), grads(odd), grads(wide), grads(dy, none, w0.clone().requires_grad_())):
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[2])
    one = torch.ones((1, 1, 1, 1), dtype=torch.bfloat16, device="cuda").expand_as(dy)
    want1 = _native.qk_norm_rope_bwd(one.contiguous(), None, base, None, w0, None)
    assert torch.equal(grads(one)[0], want1[0])
    q = base.clone().requires_grad_()
    o, _ = _native.qk_norm_rope(q, None, w0, None, out=(torch.empty_like(base), None))
    assert not o.requires_grad
    x = base.clone().requires_grad_()
    y = x * 1
    o, _ = _native.qk_norm_rope(y, None, w0, None)
    with torch.no_grad():
        y.zero_()
    with pytest.raises(RuntimeError):
        o.backward(dy)
    q, w = base.clone().requires_grad_(), w0.clone().requires_grad_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.autograd.grad(_native.qk_norm_rope(q, None, w, None)[0], (q, w), dy)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = torch.autograd.grad(_native.qk_norm_rope(q, None, w, None)[0], (q, w), dy)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[2])


def test_autograd_on_another_stream_and_without_tokens():
    """stream=: the graph's gradients are formed on that stream; empty calls give zero gradients of the weights."""
    d = 64
    g = torch.Generator().manual_seed(32)
    q0, dy = (torch.randn((2, 7, 4, d), generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    w0 = (1 + 0.3 * torch.randn(d, generator=g)).cuda()
    want = _native.qk_norm_rope_bwd(dy, None, q0, None, w0, None)
    q, w = q0.clone().requires_grad_(), w0.clone().requires_grad_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o, _ = _native.qk_norm_rope(q, None, w, None, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    o.backward(dy)
    assert torch.equal(q.grad, want[0]) and torch.equal(w.grad, want[2])
    e = torch.empty((2, 0, 4, d), dtype=torch.bfloat16, device="cuda", requires_grad=True)
    w.grad = None
    o, _ = _native.qk_norm_rope(e, None, w, None)
    o.sum().backward()
    assert e.grad.shape == e.shape and w.grad.abs().max() == 0
    assert _native.attn_get_device_status() == 0


def test_extreme_rows():
    """Rows of zeros, of the type's smallest and of large values; a row with NaN or an infinity spoils itself only."""
    d = 128
    x = torch.randn((1, 6, 1, d), generator=torch.Generator().manual_seed(3)).to(torch.bfloat16)
    x[0, 0] = 0
    x[0, 1] = 1e-38
    x[0, 2] = 1e18
    x[0, 3, 0, 5] = float("nan")
    x[0, 4, 0, 77] = float("inf")
    w = torch.ones(d)
    got, _ = _native.qk_norm_rope(x.cuda(), None, w.cuda(), None, 1e-6)
    got = got.cpu()
    y, size = S.norm_rope(x, w, 1e-6, None, False)
    fine = [0, 1, 2, 5]
    S.assert_within(got[:, fine], y[:, fine], 2.0 ** -8 * y[:, fine].abs() + 2.0 ** -20 * size[:, fine], "rows")
    assert got[0, 0].abs().max() == 0
    assert got[0, 3].isnan().all()
    assert got[0, 4, 0, 77].isnan() and (got[0, 4, 0, :77] == 0).all()   # inf * 0; the others are 0


def test_positions_out_of_range_are_reported():
    rope = _native.rope_table(10, 64)
    q = torch.randn((1, 3, 2, 64), device="cuda").to(torch.bfloat16)
    pos = torch.tensor([[-1, 4, 10]], dtype=torch.int32, device="cuda")
    got, _ = _native.qk_norm_rope(q, None, None, None, rope=rope, positions=pos)
    assert _native.attn_get_device_status() == _native.ATTN_ERR_DEVICE_ARG
    assert _native.attn_get_device_status() == 0
    ok, _ = _native.qk_norm_rope(q, None, None, None, rope=rope, positions=pos.clamp(0, 9))
    assert torch.equal(got, ok)
    assert _native.attn_get_device_status() == 0


def test_captured_and_on_another_stream():
    _, q, k, qc, kc, wq, wk, rope, pos, cs = _inputs(2, 40, 4, 2, 128, 128, 21, True, 2)
    r, p = _gpu(rope), pos.cuda()
    g = [torch.randn((2, 40, H, 128), device="cuda").to(torch.bfloat16) for H in (4, 2)]
    w = (wq.cuda(), wk.cuda())
    want = _native.qk_norm_rope(qc, kc, *w, 1e-6, r, p), _native.qk_norm_rope_bwd(*g, qc, kc, *w, 1e-6, r, p)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        two = _native.qk_norm_rope(qc, kc, *w, 1e-6, r, p), _native.qk_norm_rope_bwd(*g, qc, kc, *w, 1e-6, r, p)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        three = _native.qk_norm_rope(qc, kc, *w, 1e-6, r, p), _native.qk_norm_rope_bwd(*g, qc, kc, *w, 1e-6, r, p)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for got in (two, three):
        for a, b in zip(want[0] + want[1], got[0] + got[1]):
            assert torch.equal(a, b)


def test_a_late_stream_keeps_what_the_call_allocated():
    """stream=: what the calls allocate is that stream's, so allocations of the current stream made while the other
    is still behind do not get the workspace or outputs."""
    _, q, k, qc, kc, wq, wk, rope, pos, cs = _inputs(2, 40, 4, 2, 128, 128, 22, True, 2)
    r, p, w = _gpu(rope), pos.cuda(), (wq.cuda(), wk.cuda())
    g = [torch.randn((2, 40, H, 128), device="cuda").to(torch.bfloat16) for H in (4, 2)]
    want = _native.qk_norm_rope(qc, kc, *w, 1e-6, r, p) + _native.qk_norm_rope_bwd(*g, qc, kc, *w, 1e-6, r, p)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(50_000_000)
    got = _native.qk_norm_rope(qc, kc, *w, 1e-6, r, p, stream=side) + _native.qk_norm_rope_bwd(
        *g, qc, kc, *w, 1e-6, r, p, stream=side)
    sizes = [t.numel() * t.element_size() for t in want] + [
        _native.attn_qk_norm_rope_bwd_workspace_size(2, 40, 4, 2, 128)]
    held = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(4)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert all(bool((h == 255).all()) for h in held)


def test_refusals():
    q = torch.zeros((1, 2, 2, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, device="cuda")
    rope = _native.rope_table(8, 64)
    for bad in (lambda: _native.qk_norm_rope(q.float(), None, w, None),
                lambda: _native.qk_norm_rope(q, q, w.bfloat16(), w),
                lambda: _native.qk_norm_rope(q, q, w[:32], w),
                lambda: _native.qk_norm_rope(q, q.cpu(), w, w),
                lambda: _native.qk_norm_rope(q, q, w, w, rope=(rope[0], rope[1][:4])),
                lambda: _native.qk_norm_rope(q, q, w, w, rope=rope, positions=torch.zeros((1, 2), device="cuda")),
                lambda: _native.qk_norm_rope(q, q, w, w, out=(q[:, :1], q)),
                lambda: _native.qk_norm_rope_bwd(q, q, q, q, w, w, workspace=torch.empty(1 << 20, dtype=torch.uint8)),
                lambda: _native.qk_norm_rope_bwd(q, q, q[:, :1], q, w, w)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(_native.AttnError):
        _native.qk_norm_rope(q, q, w, w, eps=0.0)
    other = torch.zeros_like(q)
    for out in ((other, other), (other, q)):     # outputs over each other, an output over the other input
        with pytest.raises(_native.AttnError):
            _native.qk_norm_rope(q, other.clone(), w, w, out=out)
    with pytest.raises(_native.AttnError):
        _native.qk_norm_rope(q[..., :48].contiguous(), None, None, None)

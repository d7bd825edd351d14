"""Host-side argument checks of the operators around the attention kernels,
the binding's own checks, and the plain forms that the GPU tests compare with
(no GPU: every C call here returns before any CUDA call)."""
import ctypes
import math
import os
import re

import pytest
import torch

from exact_io_aware_14_gb300 import _native, build as native_build
from tests import _serving as S


@pytest.fixture(scope="module")
def L():
    native_build.build()
    return _native.lib()


def _vp(x):
    return ctypes.c_void_p(x) if x else None


def _qk(L, **kw):
    a = dict(q=16, qs=1024, k=16, ks=256, wq=16, wk=16, eps=1e-6, c=16, s=16, mp=64, rot=128, inter=0, pos=0, qo=32,
             ko=32, B=2, N=5, Hq=8, Hkv=2, d=128)
    a.update(kw)
    return L.attn_qk_norm_rope(_vp(a["q"]), a["qs"], _vp(a["k"]), a["ks"], _vp(a["wq"]), _vp(a["wk"]), a["eps"],
                               _vp(a["c"]), _vp(a["s"]), a["mp"], a["rot"], a["inter"], _vp(a["pos"]), _vp(a["qo"]),
                               _vp(a["ko"]), a["B"], a["N"], a["Hq"], a["Hkv"], a["d"], None)


@pytest.mark.parametrize("want,kw", [
    (0, dict(N=0)), (1, dict(B=0)), (1, dict(N=-1)), (1, dict(Hq=0)), (1, dict(Hkv=-1)), (2, dict(d=96)),
    (1, dict(rot=-16)), (1, dict(rot=144)), (2, dict(rot=24)), (1, dict(c=0)), (1, dict(s=0)), (1, dict(mp=0)),
    (3, dict(c=20)), (1, dict(inter=2)), (1, dict(eps=0.0)), (1, dict(eps=-1.0)), (1, dict(eps=math.nan)),
    (1, dict(q=0)), (1, dict(k=0)), (1, dict(qo=0)), (1, dict(ko=0)), (1, dict(qs=1016)), (3, dict(qs=1028)),
    (3, dict(q=24)), (3, dict(qo=40)), (3, dict(wq=20)), (3, dict(pos=18)),
    (1, dict(qo=16, qs=2048)),                # in place needs dense rows
    (2, dict(B=1 << 20, N=1 << 20)), (2, dict(Hq=1 << 21, qs=1 << 28)), (2, dict(qs=1 << 31)),
    # outputs over another tensor's rows: the other input, the other output, an input moved by one row
    (1, dict(q=1 << 20, k=2 << 20, qo=2 << 20, ko=4 << 20)), (1, dict(q=1 << 20, k=2 << 20, qo=3 << 20, ko=1 << 20)),
    (1, dict(q=1 << 20, k=2 << 20, qo=3 << 20, ko=(3 << 20) + 10 * 2048 - 16)),
    (1, dict(q=1 << 20, k=2 << 20, qo=(1 << 20) + 256, ko=3 << 20)),
])
def test_qk_norm_rope_argument_checks(L, want, kw):
    assert _qk(L, **kw) == want


def _qkb(L, **kw):
    a = dict(gq=16, gk=16, q=16, qs=1024, k=16, ks=256, wq=16, wk=16, eps=1e-6, c=16, s=16, mp=64, rot=128, inter=0,
             pos=0, dq=32, dk=32, dwq=16, dwk=16, B=2, N=5, Hq=8, Hkv=2, d=128, ws=16, wsb=1 << 24)
    a.update(kw)
    return L.attn_qk_norm_rope_bwd(_vp(a["gq"]), _vp(a["gk"]), _vp(a["q"]), a["qs"], _vp(a["k"]), a["ks"],
                                   _vp(a["wq"]), _vp(a["wk"]), a["eps"], _vp(a["c"]), _vp(a["s"]), a["mp"], a["rot"],
                                   a["inter"], _vp(a["pos"]), _vp(a["dq"]), _vp(a["dk"]), _vp(a["dwq"]),
                                   _vp(a["dwk"]), a["B"], a["N"], a["Hq"], a["Hkv"], a["d"], _vp(a["ws"]), a["wsb"],
                                   None)


@pytest.mark.parametrize("want,kw", [
    (0, dict(N=0, wq=0, wk=0, dwq=0, dwk=0)), (1, dict(B=0)), (2, dict(d=80)), (1, dict(rot=130)),
    (1, dict(eps=0.0)), (1, dict(dwq=0)), (1, dict(wk=0)), (1, dict(gq=0)), (1, dict(dk=0)), (1, dict(q=0)),
    (1, dict(ks=128)), (3, dict(ks=260)), (3, dict(gq=24)), (3, dict(dwq=18)), (7, dict(ws=0)), (7, dict(wsb=64)),
    (7, dict(ws=24)), (1, dict(Hkv=0)), (2, dict(ks=1 << 31)),
    (1, dict(gq=1 << 20, gk=2 << 20, q=3 << 20, k=4 << 20, dq=3 << 20, dk=2 << 20)),
    (1, dict(gq=1 << 20, gk=2 << 20, q=3 << 20, k=4 << 20, dq=2 << 20, dk=5 << 20)),
    (1, dict(gq=1 << 20, gk=2 << 20, q=3 << 20, k=4 << 20, dq=(1 << 20) + 256, dk=2 << 20)),
])
def test_qk_norm_rope_bwd_argument_checks(L, want, kw):
    assert _qkb(L, **kw) == want


def test_bwd_workspace_size(L):
    n = L.attn_qk_norm_rope_bwd_workspace_size(4, 4096, 32, 8, 128)
    assert 0 < n <= 16 << 20 and n % 512 == 0
    assert L.attn_qk_norm_rope_bwd_workspace_size(1, 1, 1, 0, 64) == 256
    assert L.attn_qk_norm_rope_bwd_workspace_size(0, 1, 1, 1, 64) == 0
    assert L.attn_qk_norm_rope_bwd_workspace_size(1, 1, 1, 1, 96) == 0
    assert _qkb(L, wsb=L.attn_qk_norm_rope_bwd_workspace_size(2, 5, 8, 2, 128) - 1) == 7


def _app(L, fp8=False, **kw):
    a = dict(k=16, ks=1024, v=16, vs=1024, kp=16, vp=16, sk=16, sv=16, bt=16, mb=8, ps=256, npg=64, sl=16, nl=0,
             so=0, c=16, s=16, mp=2048, rot=128, inter=0, B=2, Nn=3, Hkv=8, d=128)
    a.update(kw)
    args = [_vp(a["k"]), a["ks"], _vp(a["v"]), a["vs"], _vp(a["kp"]), _vp(a["vp"])]
    if fp8:
        args += [_vp(a["sk"]), _vp(a["sv"])]
    args += [_vp(a["bt"]), a["mb"], a["ps"], a["npg"], _vp(a["sl"]), _vp(a["nl"]), _vp(a["so"]), _vp(a["c"]),
             _vp(a["s"]), a["mp"], a["rot"], a["inter"], a["B"], a["Nn"], a["Hkv"], a["d"], None]
    return (L.attn_kvcache_append_paged_fp8 if fp8 else L.attn_kvcache_append_paged)(*args)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("want,kw", [
    (1, dict(B=0)), (1, dict(Nn=-1)), (1, dict(Hkv=0)), (1, dict(mb=0)), (1, dict(npg=0)), (1, dict(ps=0)),
    (1, dict(ps=100)), (2, dict(d=96)), (2, dict(B=65536)), (2, dict(mb=1 << 23)), (1, dict(sl=0)), (1, dict(bt=0)),
    (1, dict(kp=0)), (1, dict(vp=0)), (1, dict(so=16)), (1, dict(nl=32, so=32)),
    (1, dict(k=0)), (1, dict(v=0)), (1, dict(ks=1016)), (2, dict(ks=1 << 31)),
    (3, dict(vs=1028)), (3, dict(k=24)), (3, dict(kp=24)), (3, dict(bt=18)), (3, dict(sl=18)), (3, dict(nl=18)),
    (3, dict(so=18)), (1, dict(so=20)), (1, dict(sl=64, nl=32, so=28)), (1, dict(rot=130)), (2, dict(rot=8)), (1, dict(c=0)), (3, dict(s=24)), (1, dict(inter=-1)),
])
def test_append_argument_checks(L, fp8, want, kw):
    assert _app(L, fp8, **kw) == want


def test_append_fp8_wants_scales(L):
    assert _app(L, True, sk=0) == 1
    assert _app(L, True, sv=0) == 1
    assert _app(L, True, sv=18) == 3


def test_append_refuses_one_memory_for_keys_and_values(L):
    apart = dict(kp=1 << 30, vp=1 << 31, sk=1 << 20, sv=1 << 21)
    assert _app(L, False, **dict(apart, vp=1 << 30)) == 1
    assert _app(L, True, **dict(apart, vp=1 << 30)) == 1
    assert _app(L, True, **dict(apart, sv=1 << 20)) == 1


def _dec(L, **kw):
    a = dict(q=16, kp=16, vp=16, sk=16, sv=16, bt=16, mb=8, ps=256, npg=64, sl=16, o=16, lse=16, B=2, Nq=1, Hq=8,
             Hkv=2, d=128, scale=0.1, chunk=1024, ws=16, wsb=1 << 30)
    a.update(kw)
    return L.attn_fwd_splitkv_paged_fp8(_vp(a["q"]), _vp(a["kp"]), _vp(a["vp"]), _vp(a["sk"]), _vp(a["sv"]),
                                        _vp(a["bt"]), a["mb"], a["ps"], a["npg"], _vp(a["sl"]), _vp(a["o"]),
                                        _vp(a["lse"]), a["B"], a["Nq"], a["Hq"], a["Hkv"], a["d"], a["scale"],
                                        a["chunk"], _vp(a["ws"]), a["wsb"], None)


@pytest.mark.parametrize("want,kw", [
    (1, dict(B=0)), (1, dict(Nq=0)), (2, dict(Nq=65)), (1, dict(Hq=7)), (1, dict(mb=0)), (1, dict(npg=0)),
    (1, dict(ps=32)), (1, dict(ps=100)), (1, dict(chunk=0)), (1, dict(chunk=100)), (2, dict(chunk=2112)), (1, dict(scale=math.inf)),
    (2, dict(d=256)), (2, dict(mb=1 << 23)), (2, dict(B=65536)), (1, dict(q=0)), (1, dict(sk=0)), (1, dict(sv=0)),
    (1, dict(bt=0)), (1, dict(sl=0)), (1, dict(o=0)), (1, dict(lse=0)), (3, dict(q=24)), (3, dict(kp=24)),
    (3, dict(sk=18)), (3, dict(bt=18)), (3, dict(lse=18)), (7, dict(ws=0)), (7, dict(ws=24)), (7, dict(wsb=1024)),
    (1, dict(q=1 << 20, o=1 << 20)), (1, dict(q=1 << 20, o=(1 << 20) + 2 * 8 * 256 - 16)),
])
def test_decode_fp8_argument_checks(L, want, kw):
    assert _dec(L, **kw) == want


def test_decode_fp8_workspace_and_chunk(L):
    need = L.attn_splitkv_workspace_size(2, 3 * 8, 8 * 256, 128, 512)
    assert _dec(L, Nq=3, chunk=512, wsb=need - 1) == 7
    for B, Nq, Hq, Hkv, n in ((1, 1, 32, 8, 64), (1, 1, 32, 8, 1 << 20), (64, 7, 8, 1, 4096), (16, 1, 32, 8, 16384),
                             (65535, 64, 128, 1, 2 ** 31 - 1), (1, 1, 1, 1, 1)):
        c = L.attn_splitkv_fp8_chunk(B, Nq, Hq, Hkv, n)
        assert 64 <= c <= 2048 and c % 64 == 0
    assert L.attn_splitkv_fp8_chunk(0, 1, 8, 8, 64) == 0
    assert L.attn_splitkv_fp8_chunk(1, 1, 8, 3, 64) == 0


def test_workspace_of_the_longest_tables(L):
    """Capacities whose sum with the split length passes 31 bits."""
    n = 2 ** 31 - 1
    for chunk in (2048, 1 << 20):
        splits = -(-n // chunk)
        assert L.attn_splitkv_workspace_size(3, 2, n, 64, chunk) == 3 * 2 * splits * (64 + 1) * 4


def test_dependent_kernels_use_no_read_only_loads():
    """Kernels that start while earlier ones run must not read through the read-only path, whose loads the compiler may
    move before the wait and which wants memory that nothing writes while the kernel lives."""
    csrc = os.path.dirname(native_build.LIB.replace("_build", "csrc"))
    for name in ("qk_norm_rope_sm103.cu", "append_sm103.cu", "decode_fp8_sm103.cu", "rope.cuh", "ptx.cuh"):
        text = open(os.path.join(csrc, name)).read()
        assert not re.search(r"__ldg|ld\.global\.nc|__restrict__", text), name


def test_tensor_memory_is_asked_for_after_the_wait():
    """A kernel that starts while the one before it runs holds no Tensor Memory while it waits: that kernel may have CTAs
    that still need some, and neither would go on."""
    csrc = os.path.dirname(native_build.LIB.replace("_build", "csrc"))
    text = open(os.path.join(csrc, "decode_fp8_sm103.cu")).read()
    assert 0 < text.index("  grid_wait();") < text.index("  tmem_alloc(")


def test_binding_refuses_tensors_off_the_gpu():
    x = torch.zeros((1, 1, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        _native.qk_norm_rope(x, x, None, None)
    with pytest.raises(ValueError):
        _native.qk_norm_rope_bwd(x, x, x, x, None, None)
    with pytest.raises(ValueError):
        _native.kvcache_append_paged(x, x, x, x, x, x)
    with pytest.raises(ValueError):
        _native.decode_paged_fp8(x, x, x, x, x, x, x, 1.0)


def test_binding_refuses_workspaces_and_streams_of_other_devices():
    w = torch.zeros(64)
    assert _native._space(w, -1) == (w.data_ptr(), 256)
    for bad, dev in ((w, 0), (w[::2], -1)):
        with pytest.raises(ValueError):
            _native._space(bad, dev)

    class Stream:
        device_index = 1
    with pytest.raises(ValueError):
        _native._on(Stream(), 0)


def test_row_strides_of_parts_of_a_projection():
    """The binding reads parts of fused projections in place: their row distance, or a refusal."""
    dev = -1   # the CPU
    qkv = torch.zeros((3, 5, 12, 64), dtype=torch.bfloat16)
    rows = lambda t: _native._rows("t", t, tuple(t.shape), dev)[1]
    assert rows(qkv[:, :, :8]) == 12 * 64
    assert rows(qkv[:, :, 8:10]) == 12 * 64
    assert rows(qkv[:, :1, :8]) == 5 * 12 * 64     # one token a sequence: the batch's distance
    assert rows(qkv[:1, :1, :8]) == 8 * 64         # one token: no distance
    assert rows(qkv[:1, :, 3:4]) == 12 * 64
    assert rows(qkv) == 12 * 64
    for bad in (qkv[:, ::2, :8], qkv[:, :3, :8], qkv[:, :, ::2], qkv.transpose(1, 2), qkv[..., ::2]):
        with pytest.raises(ValueError):
            rows(bad)


def test_rope_table_far_positions():
    cos, sin = _native.rope_table(300001, 32, base=10000.0, device="cpu")
    i = torch.arange(16, dtype=torch.float64)
    a = 300000 * 10000.0 ** (-2 * i / 32)
    assert cos.shape == (300001, 16) and cos.dtype == torch.float32
    assert (cos[300000].double() - a.cos()).abs().max() < 2 ** -24
    assert (sin[300000].double() - a.sin()).abs().max() < 2 ** -24


def test_plain_scale_and_rounding():
    """The plain forms themselves: scales at and around their borders, e4m3 rounding against torch's."""
    amax = torch.tensor([0.0, 448.0, 448.5, 448.6, 1.0, 1.75, 1.7519, 1.752, 897.0, 897.1, 3e38, 1e-40]).double()
    want = [2.0 ** -100, 1.0, 1.0, 2.0, 2.0 ** -8, 2.0 ** -8, 2.0 ** -8, 2.0 ** -7, 2.0, 4.0, 2.0 ** 120, 2.0 ** -100]
    assert S.scale_for(amax).tolist() == want
    x = torch.cat([torch.randn(4096, generator=torch.Generator().manual_seed(1)) * 50,
                   torch.arange(-448, 449) / 256.0, torch.tensor([448.5, 447.9, 2.0 ** -10, 3 * 2.0 ** -10])])
    x = x.clamp(-448.5, 448.5)
    assert torch.equal(S.round_e4m3(x.double()).float(), x.to(torch.float8_e4m3fn).float())


def test_rounding_to_odd_first_gives_the_nearest_code():
    """What the append keeps between finding a page's scale and writing its codes: the fp32 value cut to bf16, the last bit
    set where anything was cut.  Rounded to e4m3 it gives the code that the value itself gives, next to every border
    between two codes and at random."""
    codes = torch.arange(0, 0x7F, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    ties = torch.cat((codes, (codes[1:] + codes[:-1]) / 2, torch.tensor([448.5, 464.0]).double())).float()
    bits = ties.view(torch.int32)[:, None] + torch.arange(-70000, 70001, 7, dtype=torch.int32)
    bits = torch.cat((bits, ties.view(torch.int32)[:, None] + torch.arange(-9, 10, dtype=torch.int32)), 1).flatten()
    x = bits[bits >= 0].view(torch.float32)
    g = torch.Generator().manual_seed(6)
    x = torch.cat((x[x <= 448.5], torch.rand(200000, generator=g) * 448, torch.randn(200000, generator=g) * 0.01))
    for v in (x, -x):
        u = v.view(torch.int32)
        odd = (u & -65536) | ((u & 0xFFFF) != 0).int() * (1 << 16)
        want = S.round_e4m3(v.double()).clamp(-448.0, 448.0)
        assert torch.equal(S.round_e4m3(odd.view(torch.float32).double()).clamp(-448.0, 448.0), want)


def test_plain_gradients_against_differences():
    """The formulas of the backward pass against central differences of the forward formula, in 64 bits."""
    g = torch.Generator().manual_seed(7)
    B, N, H, d, eps = 2, 3, 2, 64, 1e-6
    x, dy, v = (torch.randn((B, N, H, d), generator=g, dtype=torch.float64) for _ in range(3))
    w, vw = (torch.randn(d, generator=g, dtype=torch.float64) for _ in range(2))
    a = torch.randn((9, 16), generator=g, dtype=torch.float64)
    pos = torch.tensor([[3, 4, 5], [0, 8, 2]])
    for inter in (False, True):
        cs = (a.cos()[pos][:, :, None], a.sin()[pos][:, :, None])
        f = lambda x, w: (S.norm_rope(x, w, eps, cs, inter)[0] * dy).sum()
        dx, _, dw, _ = S.norm_rope_bwd(dy, x, w, eps, cs, inter)
        h = 1e-6
        assert abs(float((f(x + h * v, w) - f(x - h * v, w)) / (2 * h) - (dx * v).sum())) < 1e-6
        assert abs(float((f(x, w + h * vw) - f(x, w - h * vw)) / (2 * h) - (dw * vw).sum())) < 1e-6

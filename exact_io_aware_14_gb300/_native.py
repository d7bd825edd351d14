"""ctypes binding of libattn_sm103.so (include/attn.h).

Argument marshalling only: every step of the computation runs in the CUDA
library.  If the library has not been built, the first call raises -- there
is no fallback of any kind.
"""
import ctypes
import os
import re

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "_build", "libattn_sm103.so")
HEADER = os.path.join(os.path.dirname(HERE), "include", "attn.h")

ATTN_OK = 0
ATTN_ERR_TIMEOUT = 5
ATTN_ERR_DEVICE_ARG = 6
STATUS_NAMES = {
    0: "ATTN_OK", 1: "ATTN_ERR_INVALID_ARG", 2: "ATTN_ERR_UNSUPPORTED", 3: "ATTN_ERR_MISALIGNED",
    4: "ATTN_ERR_LAUNCH", 5: "ATTN_ERR_TIMEOUT", 6: "ATTN_ERR_DEVICE_ARG", 7: "ATTN_ERR_WORKSPACE",
}

_lib = None


class AttnError(RuntimeError):
    def __init__(self, code, what):
        self.code = code
        super().__init__("%s failed: %s (%s)" % (what, STATUS_NAMES.get(code, code), status_string(code)))


def declared_functions():
    """Names of the functions include/attn.h declares."""
    text = open(HEADER).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"^\s*(?:ATTN_API\s+)?(?:const\s+)?\w+\**\s+\**(attn_\w+)\s*\(", text, flags=re.M)))


def lib():
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("CUDA attention library not built (%s); run __graft_entry__.build()" % LIB_PATH)
        _lib = _open(LIB_PATH)
    return _lib


_variants = {}


def variant_lib(name):
    """A build variant of the library (same interface; see build.VARIANTS),
    built on first use.  Pass it as ``library=`` to the calls below."""
    if name not in _variants:
        from . import build as _build
        _variants[name] = _open(_build.build_variant(name))
    return _variants[name]


def _open(path):
    """Loads one build of the library and declares its C signatures."""
    L = ctypes.CDLL(path)
    vp, i, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    L.attn_fwd.restype = i
    L.attn_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, i, f, vp]
    L.attn_fwd_window.restype = i
    L.attn_fwd_window.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, i, i, i, f, vp]
    L.attn_fwd_kvcache.restype = i
    L.attn_fwd_kvcache.argtypes = [vp, vp, vp, vp, i, vp, vp, i, i, i, i, i, i, i, i, f, vp]
    L.attn_splitkv_workspace_size.restype = sz
    L.attn_splitkv_workspace_size.argtypes = [i, i, i, i, i]
    L.attn_fwd_splitkv.restype = i
    L.attn_fwd_splitkv.argtypes = [vp, vp, vp, vp, i, vp, vp, i, i, i, i, f, i, vp, sz, vp]
    L.attn_fwd_splitkv_paged.restype = i
    L.attn_fwd_splitkv_paged.argtypes = [vp, vp, vp, vp, i, i, i, vp, vp, vp, i, i, i, i, f, i, vp, sz, vp]
    L.attn_fwd_splitkv_noalloc.restype = i
    L.attn_fwd_splitkv_noalloc.argtypes = [vp, vp, vp, vp, i, vp, vp, i, i, i, i, f, i, vp]
    ll = ctypes.c_longlong
    L.attn_qk_norm_rope.restype = i
    L.attn_qk_norm_rope.argtypes = [vp, ll, vp, ll, vp, vp, f, vp, vp, i, i, i, vp, vp, vp, i, i, i, i, i, vp]
    L.attn_qk_norm_rope_bwd_workspace_size.restype = sz
    L.attn_qk_norm_rope_bwd_workspace_size.argtypes = [i, i, i, i, i]
    L.attn_qk_norm_rope_bwd.restype = i
    L.attn_qk_norm_rope_bwd.argtypes = [vp, vp, vp, ll, vp, ll, vp, vp, f, vp, vp, i, i, i, vp, vp, vp, vp, vp,
                                        i, i, i, i, i, vp, sz, vp]
    append = [vp, ll, vp, ll, vp, vp, vp, i, i, i, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, vp]
    L.attn_kvcache_append_paged.restype = i
    L.attn_kvcache_append_paged.argtypes = append
    L.attn_kvcache_append_paged_fp8.restype = i
    L.attn_kvcache_append_paged_fp8.argtypes = append[:6] + [vp, vp] + append[6:]
    L.attn_splitkv_fp8_chunk.restype = i
    L.attn_splitkv_fp8_chunk.argtypes = [i, i, i, i, i]
    L.attn_fwd_splitkv_paged_fp8.restype = i
    L.attn_fwd_splitkv_paged_fp8.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, vp, vp, vp, i, i, i, i, i, f, i, vp, sz,
                                             vp]
    L.attn_kvcache_reserve_paged.restype = i
    L.attn_kvcache_reserve_paged.argtypes = [vp, i, i, i, vp, vp, vp, vp, vp, vp, vp, vp, i, i, vp]
    L.attn_kvcache_release_paged.restype = i
    L.attn_kvcache_release_paged.argtypes = [vp, i, i, i, vp, vp, vp, vp, vp, i, vp]
    L.attn_splitkv_paged_shared_workspace_size.restype = sz
    L.attn_splitkv_paged_shared_workspace_size.argtypes = [i, i, i, i, i]
    L.attn_fwd_splitkv_paged_shared.restype = i
    L.attn_fwd_splitkv_paged_shared.argtypes = [vp, vp, vp, vp, i, i, i, vp, i, vp, vp, i, i, i, i, i, f, vp, sz, vp]
    L.attn_kvcache_bounds_paged.restype = i
    L.attn_kvcache_bounds_paged.argtypes = [vp, vp, vp, i, i, i, vp, vp, i, i, i, i, vp]
    L.attn_select_blocks_workspace_size.restype = sz
    L.attn_select_blocks_workspace_size.argtypes = [i, i, i, i]
    L.attn_select_blocks_paged.restype = i
    L.attn_select_blocks_paged.argtypes = [vp, vp, vp, i, i, i, vp, vp, i, i, i, i, i, i, i, i, vp, sz, vp]
    L.attn_fwd_blocks_paged_workspace_size.restype = sz
    L.attn_fwd_blocks_paged_workspace_size.argtypes = [i, i, i, i, i, i, i]
    L.attn_fwd_blocks_paged.restype = i
    L.attn_fwd_blocks_paged.argtypes = [vp, vp, vp, vp, i, i, i, vp, vp, i, vp, vp, i, i, i, i, i, f, vp, sz, vp]
    L.attn_get_device_status.restype = i
    L.attn_get_device_status.argtypes = [vp]
    L.attn_selftest_wait_timeout.restype = i
    L.attn_selftest_wait_timeout.argtypes = [ctypes.c_ulonglong, vp]
    L.attn_status_string.restype = ctypes.c_char_p
    L.attn_status_string.argtypes = [i]
    L.attn_selftest_exp2_poly.restype = i
    L.attn_selftest_exp2_poly.argtypes = [vp, vp, ctypes.c_longlong, vp]
    L.attn_probe_read_bandwidth.restype = i
    L.attn_probe_read_bandwidth.argtypes = [vp, sz, vp, vp]
    return L


def status_string(code: int) -> str:
    return lib().attn_status_string(int(code)).decode()


def _stream_handle(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def _check_bf16(name, t, shape):
    if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous() or tuple(t.shape) != tuple(shape):
        raise ValueError("%s must be a contiguous CUDA bf16 tensor of shape %s (got %s %s %s)"
                         % (name, tuple(shape), t.dtype, tuple(t.shape), t.device))


# --------------------------------------------------------------------------- raw entry points
def _check_prefill(q, k, v, o, lse):
    B, Nq, Hq, d = q.shape
    Nk, Hkv = k.shape[1], k.shape[2]
    _check_bf16("q", q, (B, Nq, Hq, d))
    _check_bf16("k", k, (B, Nk, Hkv, d))
    _check_bf16("v", v, (B, Nk, Hkv, d))
    _check_bf16("o", o, (B, Nq, Hq, d))
    if lse.dtype != torch.float32 or not lse.is_cuda or not lse.is_contiguous() or tuple(lse.shape) != (B, Hq, Nq):
        raise ValueError("lse must be a contiguous CUDA fp32 tensor of shape %s" % ((B, Hq, Nq),))
    return B, Hq, Hkv, Nq, Nk, d


def _window(window):
    """None or (left, right); a negative side is unbounded."""
    if window is None:
        return -1, -1
    wl, wr = (int(x) for x in window)
    return wl, wr


def attn_fwd(q, k, v, o, lse, causal, scale, stream=None, library=None):
    """Same contract as the C call: writes o [B,Nq,Hq,d] and lse [B,Hq,Nq]. Returns the status.
    library: a build variant from variant_lib(), else the default build."""
    B, Hq, Hkv, Nq, Nk, d = _check_prefill(q, k, v, o, lse)
    return (library or lib()).attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, Hq, Hkv, Nq, Nk, d,
                                       int(causal), float(scale), _stream_handle(stream))


def attn_fwd_window(q, k, v, o, lse, causal, window, scale, stream=None):
    """attn_fwd with a local window (left, right), aligned bottom-right. Returns the status."""
    B, Hq, Hkv, Nq, Nk, d = _check_prefill(q, k, v, o, lse)
    wl, wr = _window(window)
    return lib().attn_fwd_window(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, Hq, Hkv, Nq, Nk, d,
                                 int(causal), wl, wr, float(scale), _stream_handle(stream))


def attn_fwd_kvcache(q, k_cache, v_cache, seqlens, o, lse, causal, scale, stream=None, window=None):
    """Same contract as the C call: q, o [B,Nq,Hq,d]; caches [B,max_seqlen,Hkv,d];
    seqlens int32 [B] on the device; lse [B,Hq,Nq].  Returns the status."""
    B, Nq, Hq, d = q.shape
    max_seqlen, Hkv = k_cache.shape[1], k_cache.shape[2]
    _check_bf16("q", q, (B, Nq, Hq, d))
    _check_bf16("k_cache", k_cache, (B, max_seqlen, Hkv, d))
    _check_bf16("v_cache", v_cache, (B, max_seqlen, Hkv, d))
    _check_bf16("o", o, (B, Nq, Hq, d))
    if seqlens.dtype != torch.int32 or not seqlens.is_cuda or tuple(seqlens.shape) != (B,):
        raise ValueError("seqlens must be a CUDA int32 tensor of shape (%d,)" % B)
    if lse.dtype != torch.float32 or not lse.is_cuda or not lse.is_contiguous() or tuple(lse.shape) != (B, Hq, Nq):
        raise ValueError("lse must be a contiguous CUDA fp32 tensor of shape %s" % ((B, Hq, Nq),))
    wl, wr = _window(window)
    return lib().attn_fwd_kvcache(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(seqlens), max_seqlen, _ptr(o),
                                  _ptr(lse), B, Hq, Hkv, Nq, d, int(causal), wl, wr, float(scale),
                                  _stream_handle(stream))


def forward_kvcache(q, k_cache, v_cache, seqlens, causal, scale, stream=None, window=None):
    """Allocates O and LSE and runs attn_fwd_kvcache. Returns (o, lse)."""
    B, Nq, Hq, d = q.shape
    o = torch.empty_like(q)
    lse = torch.empty((B, Hq, Nq), dtype=torch.float32, device=q.device)
    rc = attn_fwd_kvcache(q, k_cache, v_cache, seqlens, o, lse, causal, scale, stream, window)
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_fwd_kvcache")
    return o, lse


def attn_splitkv_workspace_size(B, Hq, max_seqlen, d, chunk):
    return int(lib().attn_splitkv_workspace_size(B, Hq, max_seqlen, d, chunk))


def attn_fwd_splitkv(q, k_cache, v_cache, seqlens, o, lse, scale, chunk, workspace, stream=None):
    """Same contract as the C call. workspace: a CUDA uint8 tensor. Returns the status."""
    B, _, Hq, d = q.shape
    max_seqlen, Hkv = k_cache.shape[1], k_cache.shape[2]
    _check_bf16("q", q, (B, 1, Hq, d))
    _check_bf16("k_cache", k_cache, (B, max_seqlen, Hkv, d))
    _check_bf16("v_cache", v_cache, (B, max_seqlen, Hkv, d))
    _check_bf16("o", o, (B, 1, Hq, d))
    if seqlens.dtype != torch.int32 or not seqlens.is_cuda or tuple(seqlens.shape) != (B,):
        raise ValueError("seqlens must be a CUDA int32 tensor of shape (%d,)" % B)
    if lse.dtype != torch.float32 or not lse.is_cuda or tuple(lse.shape) != (B, Hq, 1):
        raise ValueError("lse must be a CUDA fp32 tensor of shape %s" % ((B, Hq, 1),))
    return lib().attn_fwd_splitkv(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(seqlens), max_seqlen,
                                  _ptr(o), _ptr(lse), B, Hq, Hkv, d, float(scale), int(chunk),
                                  _ptr(workspace), workspace.numel() * workspace.element_size(),
                                  _stream_handle(stream))


def attn_fwd_splitkv_paged(q, k_pages, v_pages, block_table, seqlens, o, lse, scale, chunk, workspace, stream=None):
    """Same contract as the C call: k_pages, v_pages [num_pages, page_size, Hkv, d];
    block_table int32 [B, max_blocks] on the device.  Returns the status."""
    B, _, Hq, d = q.shape
    num_pages, page_size, Hkv = k_pages.shape[0], k_pages.shape[1], k_pages.shape[2]
    max_blocks = block_table.shape[1]
    _check_bf16("q", q, (B, 1, Hq, d))
    _check_bf16("k_pages", k_pages, (num_pages, page_size, Hkv, d))
    _check_bf16("v_pages", v_pages, (num_pages, page_size, Hkv, d))
    _check_bf16("o", o, (B, 1, Hq, d))
    if block_table.dtype != torch.int32 or not block_table.is_cuda or not block_table.is_contiguous() \
            or tuple(block_table.shape) != (B, max_blocks):
        raise ValueError("block_table must be a contiguous CUDA int32 tensor of shape (%d, max_blocks)" % B)
    if seqlens.dtype != torch.int32 or not seqlens.is_cuda or tuple(seqlens.shape) != (B,):
        raise ValueError("seqlens must be a CUDA int32 tensor of shape (%d,)" % B)
    if lse.dtype != torch.float32 or not lse.is_cuda or tuple(lse.shape) != (B, Hq, 1):
        raise ValueError("lse must be a CUDA fp32 tensor of shape %s" % ((B, Hq, 1),))
    return lib().attn_fwd_splitkv_paged(_ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(block_table), max_blocks,
                                        page_size, num_pages, _ptr(seqlens), _ptr(o), _ptr(lse), B, Hq, Hkv, d,
                                        float(scale), int(chunk), _ptr(workspace),
                                        workspace.numel() * workspace.element_size(), _stream_handle(stream))


def attn_fwd_splitkv_noalloc(q, k_cache, v_cache, seqlens, o, lse, scale, chunk, stream=None):
    """attn_fwd_splitkv without a workspace: the library's fixed device scratch
    holds the partials, so nothing is allocated (for callers that cannot
    allocate device memory).  Returns the status."""
    B, _, Hq, d = q.shape
    max_seqlen, Hkv = k_cache.shape[1], k_cache.shape[2]
    _check_bf16("q", q, (B, 1, Hq, d))
    _check_bf16("k_cache", k_cache, (B, max_seqlen, Hkv, d))
    _check_bf16("v_cache", v_cache, (B, max_seqlen, Hkv, d))
    _check_bf16("o", o, (B, 1, Hq, d))
    if seqlens.dtype != torch.int32 or not seqlens.is_cuda or tuple(seqlens.shape) != (B,):
        raise ValueError("seqlens must be a CUDA int32 tensor of shape (%d,)" % B)
    if lse.dtype != torch.float32 or not lse.is_cuda or tuple(lse.shape) != (B, Hq, 1):
        raise ValueError("lse must be a CUDA fp32 tensor of shape %s" % ((B, Hq, 1),))
    return lib().attn_fwd_splitkv_noalloc(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(seqlens), max_seqlen,
                                          _ptr(o), _ptr(lse), B, Hq, Hkv, d, float(scale), int(chunk),
                                          _stream_handle(stream))


# --------------------------------------------------------------------------- operators around the attention kernels
# These calls are launched once or more a layer and token, where the host's time for a call counts: each argument is
# looked at once, with the cheapest query that settles it, and the stream is asked for as a handle.  With `stream`, what
# a call allocates belongs to that stream; the caller keeps the tensors it passes until the stream has passed the call.
_BF16, _F32, _I32, _E4M3 = torch.bfloat16, torch.float32, torch.int32, torch.float8_e4m3fn
_fns = {}


def _fn(name):
    f = _fns.get(name)
    if f is None:
        f = _fns[name] = getattr(lib(), name)
    return f


def _call(name, dev, stream, *args):
    """The C call `name` on device number dev, whichever is current, on `stream` (None: that device's current stream).
    Raises unless it returns ATTN_OK."""
    handle = torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream
    if torch._C._cuda_getDevice() == dev:
        rc = _fn(name)(*args, handle)
    else:
        with torch.cuda.device(dev):
            rc = _fn(name)(*args, handle)
    if rc != ATTN_OK:
        raise AttnError(rc, name)


def _on(stream, dev):
    """Makes `stream` current for a call that allocates: what it allocates is then that stream's, not reused before
    the stream has passed the call."""
    if stream.device_index != dev:
        raise ValueError("the stream is one of cuda:%d, the tensors are on cuda:%d" % (stream.device_index, dev))
    return torch.cuda.stream(stream)


def _space(workspace, dev):
    """(address, bytes) of a workspace that the caller brought."""
    if workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on cuda:%d (got one on %s)" % (dev, workspace.device))
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _need(name, t, dtype, shape, dev):
    """t is a contiguous tensor of this type and shape on device number dev (-1: the CPU); returns its address."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        raise ValueError("%s must be a contiguous %s tensor of shape %s on %s (got %s %s %s)"
                         % (name, dtype, tuple(shape), "cuda:%d" % dev, t.dtype, tuple(t.shape), t.device))
    return t.data_ptr()


def _rows(name, t, shape, dev):
    """t [B, N, H, d] bf16 with dense heads and one distance between its token rows (a part of a fused projection's
    rows); returns (address, that distance)."""
    if t.dtype is not _BF16 or t.shape != shape or t.get_device() != dev:
        raise ValueError("%s must be a bf16 tensor of shape %s on %s (got %s %s %s)"
                         % (name, tuple(shape), "cuda:%d" % dev, t.dtype, tuple(t.shape), t.device))
    B, N, H, d = shape
    if t.is_contiguous():
        return t.data_ptr(), H * d
    sb, sn, sh, sd = t.stride()
    row = sn if N > 1 else (sb if B > 1 else H * d)  # distance of neighbouring tokens, whatever sizes of one say
    if sd != 1 or (sh != d and H > 1) or (N > 1 and B > 1 and sb != N * sn):
        raise ValueError("%s must have dense heads and evenly spaced token rows (strides %s)" % (name, t.stride()))
    return t.data_ptr(), row


def _rope_args(rope, interleaved, dev):
    """(cos, sin, max_pos, rot_dim, interleaved) of the C calls; rope: None or (cos, sin) fp32 [max_pos, rot_dim/2]."""
    if rope is None:
        return None, None, 0, 0, 0
    cos, sin = rope
    shape = cos.shape
    if len(shape) != 2:
        raise ValueError("rope tables must be [max_pos, rot_dim / 2]")
    return (_need("rope cos", cos, _F32, shape, dev), _need("rope sin", sin, _F32, shape, dev), shape[0],
            2 * shape[1], 1 if interleaved else 0)


def _cuda_device(t):
    dev = t.get_device()
    if dev < 0:
        raise ValueError("a CUDA tensor is wanted (got %s)" % t.device)
    return dev


def rope_table(max_pos, rot_dim, base=10000.0, device="cuda"):
    """Tables (cos, sin) fp32 [max_pos, rot_dim / 2] of the rotation by t * base^(-2i / rot_dim); the angles are
    formed in 64 bits, so those of far positions keep their accuracy."""
    inv = float(base) ** (-torch.arange(0, rot_dim, 2, dtype=torch.float64, device=device) / rot_dim)
    a = torch.arange(max_pos, dtype=torch.float64, device=device)[:, None] * inv
    return a.cos().float(), a.sin().float()


def _weight(name, w, d, dev):
    return None if w is None else _need(name, w, _F32, (d,), dev)


def qk_norm_rope(q, k, q_weight, k_weight, eps=1e-6, rope=None, positions=None, interleaved=False, out=None,
                 stream=None):
    """Norms of q and k for each head (weights fp32 [d]; None: no norm) and the position rotation, in one pass
    (attn_qk_norm_rope).  q [B,N,Hq,d], k [B,N,Hkv,d] (or None) bf16, possibly parts of a fused projection's rows;
    rope: (cos, sin) from rope_table, or None; positions int32 [B,N], or None for 0 .. N-1; out: (q_out, k_out) to
    write to (q and k themselves where dense), or None.  Returns (q_out, k_out).  Differentiable in q, k and the weights
    (qk_norm_rope_bwd runs in the backward pass); with out, no graph is recorded.  To capture a backward pass, capture its
    forward pass with it, and keep no other graph of the same leaves, as for any torch operator."""
    dev = _cuda_device(q)
    if stream is not None:
        with _on(stream, dev):
            return qk_norm_rope(q, k, q_weight, k_weight, eps, rope, positions, interleaved, out)
    if (q.requires_grad or (k is not None and k.requires_grad) or (q_weight is not None and q_weight.requires_grad)
            or (k_weight is not None and k_weight.requires_grad)) and out is None and torch.is_grad_enabled():
        return _QkNormRope.apply(q, k, q_weight, k_weight, eps, rope, positions, interleaved)
    q_shape = q.shape
    B, N, Hq, d = q_shape
    Hkv = 0 if k is None else k.shape[2]
    k_shape = (B, N, Hkv, d)
    qp, qs = _rows("q", q, q_shape, dev)
    kp, ks = (None, 0) if k is None else _rows("k", k, k_shape, dev)
    if out is None:
        qo = torch.empty(q_shape, dtype=_BF16, device=dev)
        ko = None if k is None else torch.empty(k_shape, dtype=_BF16, device=dev)
    else:
        qo, ko = out
        _need("q_out", qo, _BF16, q_shape, dev)
        if k is not None:
            _need("k_out", ko, _BF16, k_shape, dev)
    pos = None if positions is None else _need("positions", positions, _I32, (B, N), dev)
    _call("attn_qk_norm_rope", dev, stream, qp, qs, kp, ks, _weight("q_weight", q_weight, d, dev),
          _weight("k_weight", k_weight, d, dev), eps, *_rope_args(rope, interleaved, dev), pos, qo.data_ptr(),
          None if ko is None else ko.data_ptr(), B, N, Hq, Hkv, d)
    return qo, ko


class _QkNormRope(torch.autograd.Function):
    """qk_norm_rope as a node of the autograd graph."""

    @staticmethod
    def forward(ctx, q, k, q_weight, k_weight, eps, rope, positions, interleaved):
        outs = qk_norm_rope(q, k, q_weight, k_weight, eps, rope, positions, interleaved)
        if k is None or k.shape[2] == 0:
            k_weight = None   # there is nothing to differentiate
        cos, sin = (None, None) if rope is None else rope
        # without a norm x does not enter its gradient
        ctx.save_for_backward(None if q_weight is None else q, None if k_weight is None else k, q_weight, k_weight,
                              cos, sin, positions)
        ctx.eps, ctx.interleaved = eps, interleaved
        return outs

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dq_out, dk_out):
        q, k, q_weight, k_weight, cos, sin, positions = ctx.saved_tensors
        grads = qk_norm_rope_bwd(_dense(dq_out), None if dk_out is None else _dense(dk_out), q, k, q_weight, k_weight,
                                 ctx.eps, None if cos is None else (cos, sin), positions, ctx.interleaved)
        return (*grads, None, None, None, None)


def _dense(t):
    """t as the C calls want a tensor: contiguous, from a 16-byte boundary on."""
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


def attn_qk_norm_rope_bwd_workspace_size(B, N, Hq, Hkv, d):
    return int(lib().attn_qk_norm_rope_bwd_workspace_size(B, N, Hq, Hkv, d))


def qk_norm_rope_bwd(dq_out, dk_out, q, k, q_weight, k_weight, eps=1e-6, rope=None, positions=None,
                     interleaved=False, workspace=None, stream=None):
    """Gradients of qk_norm_rope (attn_qk_norm_rope_bwd): dq_out, dk_out are the gradients of its outputs, the other
    arguments its own (q, k may be None without a norm).  Returns (dq, dk, dq_weight, dk_weight), None where there
    is nothing to differentiate."""
    dev = _cuda_device(dq_out)
    if stream is not None:
        with _on(stream, dev):
            return qk_norm_rope_bwd(dq_out, dk_out, q, k, q_weight, k_weight, eps, rope, positions, interleaved,
                                    workspace)
    B, N, Hq, d = dq_out.shape
    Hkv = 0 if dk_out is None else dk_out.shape[2]
    gq = _need("dq_out", dq_out, _BF16, (B, N, Hq, d), dev)
    gk = None if dk_out is None else _need("dk_out", dk_out, _BF16, (B, N, Hkv, d), dev)
    qp, qs = (None, 0) if q_weight is None else _rows("q", q, (B, N, Hq, d), dev)
    kp, ks = (None, 0) if k_weight is None else _rows("k", k, (B, N, Hkv, d), dev)
    dq = torch.empty((B, N, Hq, d), dtype=_BF16, device=dev)
    dk = None if dk_out is None else torch.empty((B, N, Hkv, d), dtype=_BF16, device=dev)
    dwq = None if q_weight is None else torch.empty((d,), dtype=_F32, device=dev)
    dwk = None if k_weight is None else torch.empty((d,), dtype=_F32, device=dev)
    ws, nbytes = None, 0
    if dwq is not None or dwk is not None:
        if workspace is None:
            nbytes = _fn("attn_qk_norm_rope_bwd_workspace_size")(B, N, Hq, Hkv, d)
            workspace = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=dev)
        ws, nbytes = _space(workspace, dev)
    pos = None if positions is None else _need("positions", positions, _I32, (B, N), dev)
    _call("attn_qk_norm_rope_bwd", dev, stream, gq, gk, qp, qs, kp, ks, _weight("q_weight", q_weight, d, dev),
          _weight("k_weight", k_weight, d, dev), eps, *_rope_args(rope, interleaved, dev), pos, dq.data_ptr(),
          None if dk is None else dk.data_ptr(), None if dwq is None else dwq.data_ptr(),
          None if dwk is None else dwk.data_ptr(), B, N, Hq, Hkv, d, ws, nbytes)
    return dq, dk, dwq, dwk


def _append(name, k, v, k_pages, v_pages, scales, block_table, seqlens, rope, interleaved, new_lens, seqlens_out,
            stream):
    dev = _cuda_device(k_pages)
    shape = k.shape
    B, Nn, Hkv, d = shape
    pools = k_pages.shape
    num_pages, page_size = pools[:2]
    if pools[2:] != (Hkv, d):
        raise ValueError("k_pages must be [num_pages, page_size, %d, %d] (got %s)" % (Hkv, d, tuple(pools)))
    kp, ks = _rows("k", k, shape, dev)
    vp, vs = _rows("v", v, shape, dev)
    dtype = _E4M3 if scales else _BF16
    args = [kp, ks, vp, vs, _need("k_pages", k_pages, dtype, pools, dev), _need("v_pages", v_pages, dtype, pools, dev)]
    for what, s in zip(("k_scales", "v_scales"), scales):
        args.append(_need(what, s, _F32, (num_pages, Hkv), dev))
    max_blocks = block_table.shape[-1]
    _call(name, dev, stream, *args, _need("block_table", block_table, _I32, (B, max_blocks), dev), max_blocks,
          page_size, num_pages, _need("seqlens", seqlens, _I32, (B,), dev),
          None if new_lens is None else _need("new_lens", new_lens, _I32, (B,), dev),
          None if seqlens_out is None else _need("seqlens_out", seqlens_out, _I32, (B,), dev),
          *_rope_args(rope, interleaved, dev), B, Nn, Hkv, d)


def kvcache_append_paged(k, v, k_pages, v_pages, block_table, seqlens, rope=None, interleaved=False, new_lens=None,
                         seqlens_out=None, stream=None):
    """Appends new tokens' keys (rotated to their position if rope = (cos, sin) is given) and values
    [B,Nn,Hkv,d] bf16 to a paged bf16 cache in place (attn_kvcache_append_paged); seqlens int32 [B]: the lengths
    before; new_lens int32 [B]: the real ones of the Nn rows; seqlens_out int32 [B]: receives the lengths after."""
    _append("attn_kvcache_append_paged", k, v, k_pages, v_pages, (), block_table, seqlens, rope, interleaved,
            new_lens, seqlens_out, stream)


def kvcache_append_paged_fp8(k, v, k_pages, v_pages, k_scales, v_scales, block_table, seqlens, rope=None,
                             interleaved=False, new_lens=None, seqlens_out=None, stream=None):
    """kvcache_append_paged for float8_e4m3fn pages with fp32 scales [num_pages, Hkv], both updated in place
    (attn_kvcache_append_paged_fp8)."""
    _append("attn_kvcache_append_paged_fp8", k, v, k_pages, v_pages, (k_scales, v_scales), block_table, seqlens,
            rope, interleaved, new_lens, seqlens_out, stream)


def attn_splitkv_fp8_chunk(B, Nq, Hq, Hkv, max_seqlen):
    return int(lib().attn_splitkv_fp8_chunk(B, Nq, Hq, Hkv, max_seqlen))


def decode_paged_fp8(q, k_pages, v_pages, k_scales, v_scales, block_table, seqlens, scale, chunk=None,
                     workspace=None, stream=None):
    """Attention of the last Nq tokens q [B,Nq,Hq,d] bf16 of each sequence over a paged float8_e4m3fn cache with
    fp32 scales [num_pages, Hkv] (attn_fwd_splitkv_paged_fp8); chunk None: attn_splitkv_fp8_chunk's for the table's
    capacity (one for the longest sequence suits short sequences in a wide table better).
    Returns (o, lse [B,Hq,Nq])."""
    dev = _cuda_device(q)
    if stream is not None:
        with _on(stream, dev):
            return decode_paged_fp8(q, k_pages, v_pages, k_scales, v_scales, block_table, seqlens, scale, chunk,
                                    workspace)
    q_shape, pools = q.shape, k_pages.shape
    B, Nq, Hq, d = q_shape
    num_pages, page_size, Hkv = pools[:3]
    if pools[3:] != (d,):
        raise ValueError("k_pages must be [num_pages, page_size, Hkv, %d] (got %s)" % (d, tuple(pools)))
    max_blocks = block_table.shape[-1]
    args = (_need("q", q, _BF16, q_shape, dev), _need("k_pages", k_pages, _E4M3, pools, dev),
            _need("v_pages", v_pages, _E4M3, pools, dev), _need("k_scales", k_scales, _F32, (num_pages, Hkv), dev),
            _need("v_scales", v_scales, _F32, (num_pages, Hkv), dev),
            _need("block_table", block_table, _I32, (B, max_blocks), dev), max_blocks, page_size, num_pages,
            _need("seqlens", seqlens, _I32, (B,), dev))
    cap = min(max_blocks * page_size, 0x7fffffff)  # the C call refuses more
    if chunk is None:
        chunk = _fn("attn_splitkv_fp8_chunk")(B, Nq, Hq, Hkv, cap)
    o = torch.empty(q_shape, dtype=_BF16, device=dev)
    lse = torch.empty((B, Hq, Nq), dtype=_F32, device=dev)
    if workspace is None:
        n = _fn("attn_splitkv_workspace_size")(B, Nq * Hq, cap, d, chunk)
        workspace = torch.empty(n if n > 16 else 16, dtype=torch.uint8, device=dev)
    ws, n = _space(workspace, dev)
    _call("attn_fwd_splitkv_paged_fp8", dev, stream, *args, o.data_ptr(), lse.data_ptr(), B, Nq, Hq, Hkv, d,
          scale, chunk, ws, n)
    return o, lse


# --------------------------------------------------------------------------- operators on a paged cache
def _table(block_table, seqlens, B, dev):
    """(block_table, max_blocks, seqlens) as the C calls take them."""
    max_blocks = block_table.shape[-1]
    return (_need("block_table", block_table, _I32, (B, max_blocks), dev), max_blocks,
            _need("seqlens", seqlens, _I32, (B,), dev))


def kvcache_reserve_paged(block_table, seqlens, new_lens, free_pages, free_count, page_size, max_new, slots=True,
                          seqlens_out=None, stream=None):
    """Gives the sequences pages for their new tokens, on the GPU (attn_kvcache_reserve_paged): block_table int32
    [B, max_blocks] is extended in place from the stack free_pages int32 [num_pages] with free_count int32 [1] valid
    entries; seqlens int32 [B]: the tokens held; new_lens int32 [B]: how many more, at most max_new each (None: max_new
    each); seqlens_out int32 [B]: receives the lengths with the new tokens.  Returns (granted int32 [B]: new_lens, 0
    where the pages ran out, new slots int64 [B, max_new] of the tokens or None with slots=False, and the count of free
    pages that remain, int32 [1])."""
    dev = _cuda_device(block_table)
    if stream is not None:
        with _on(stream, dev):
            return kvcache_reserve_paged(block_table, seqlens, new_lens, free_pages, free_count, page_size, max_new,
                                         slots, seqlens_out)
    B, num_pages = block_table.shape[0], free_pages.shape[0]
    bt, max_blocks, sl = _table(block_table, seqlens, B, dev)
    args = (None if new_lens is None else _need("new_lens", new_lens, _I32, (B,), dev),
            _need("free_pages", free_pages, _I32, (num_pages,), dev),
            _need("free_count", free_count, _I32, (1,), dev))
    so = None if seqlens_out is None else _need("seqlens_out", seqlens_out, _I32, (B,), dev)
    granted = torch.empty((B,), dtype=_I32, device=dev)
    slot = torch.empty((B, max_new), dtype=torch.int64, device=dev) if slots else None
    count = torch.empty((1,), dtype=_I32, device=dev)
    _call("attn_kvcache_reserve_paged", dev, stream, bt, max_blocks, page_size, num_pages, sl, *args,
          granted.data_ptr(), so, None if slot is None else slot.data_ptr(), count.data_ptr(), B, max_new)
    return granted, slot, count


def kvcache_release_paged(block_table, seqlens, keep_lens, free_pages, free_count, page_size, stream=None):
    """Puts the pages behind the first keep_lens[b] of each sequence's seqlens[b] tokens back on the stack free_pages,
    in place (attn_kvcache_release_paged).  Returns the new count of free pages, int32 [1]."""
    dev = _cuda_device(block_table)
    if stream is not None:
        with _on(stream, dev):
            return kvcache_release_paged(block_table, seqlens, keep_lens, free_pages, free_count, page_size)
    B, num_pages = block_table.shape[0], free_pages.shape[0]
    bt, max_blocks, sl = _table(block_table, seqlens, B, dev)
    args = (_need("keep_lens", keep_lens, _I32, (B,), dev), _need("free_pages", free_pages, _I32, (num_pages,), dev),
            _need("free_count", free_count, _I32, (1,), dev))
    count = torch.empty((1,), dtype=_I32, device=dev)
    _call("attn_kvcache_release_paged", dev, stream, bt, max_blocks, page_size, num_pages, sl, *args,
          count.data_ptr(), B)
    return count


def _pools(q, k_pages, v_pages, block_table, seqlens, dev):
    """The arguments that the attention calls over a paged bf16 cache share, and (page_size, Hkv)."""
    B, Nq, Hq, d = q.shape
    pools = k_pages.shape
    if len(pools) != 4 or pools[3] != d:
        raise ValueError("k_pages must be [num_pages, page_size, Hkv, %d] (got %s)" % (d, tuple(pools)))
    bt, max_blocks, sl = _table(block_table, seqlens, B, dev)
    return (_need("q", q, _BF16, q.shape, dev), _need("k_pages", k_pages, _BF16, pools, dev),
            _need("v_pages", v_pages, _BF16, pools, dev), bt, max_blocks, pools[1], pools[0], sl), pools[2]


def _attend(name, size, q, pools, Hkv, extra, scale, workspace, dev, *sizes):
    B, Nq, Hq, d = q.shape
    o = torch.empty(q.shape, dtype=_BF16, device=dev)
    lse = torch.empty((B, Hq, Nq), dtype=_F32, device=dev)
    if workspace is None:
        n = _fn(size)(B, Nq, Hq, Hkv, d, *sizes)
        workspace = torch.empty(n if n > 16 else 16, dtype=torch.uint8, device=dev)
    ws, n = _space(workspace, dev)
    _call(name, dev, None, *pools, *extra, o.data_ptr(), lse.data_ptr(), B, Nq, Hq, Hkv, d, scale, ws, n)
    return o, lse


def decode_paged_shared(q, k_pages, v_pages, block_table, seqlens, shared_len, scale, workspace=None, stream=None):
    """Attention of the last Nq tokens q [B,Nq,Hq,d] bf16 of each sequence over a paged bf16 cache whose first
    shared_len keys (whole pages) all sequences have in common, the pages of row 0 of the block table
    (attn_fwd_splitkv_paged_shared).  Row i is the token at position seqlens - Nq + i: fewer new tokens than Nq are the
    last rows of q, where kvcache_append_paged takes the first ones.  Returns (o, lse [B,Hq,Nq])."""
    dev = _cuda_device(q)
    if stream is not None:
        with _on(stream, dev):
            return decode_paged_shared(q, k_pages, v_pages, block_table, seqlens, shared_len, scale, workspace)
    pools, Hkv = _pools(q, k_pages, v_pages, block_table, seqlens, dev)
    return _attend("attn_fwd_splitkv_paged_shared", "attn_splitkv_paged_shared_workspace_size", q, pools, Hkv,
                   (shared_len,), scale, workspace, dev)


def kvcache_bounds_paged(k_pages, k_bounds, block_table, seqlens, max_new, new_lens=None, stream=None):
    """Smallest and largest keys of the 64-key blocks that the last new_lens[b] (int32 [B]; None: max_new) of each
    sequence's seqlens[b] tokens reach, into k_bounds [num_pages, page_size / 64, Hkv, 2, d] bf16 in place
    (attn_kvcache_bounds_paged)."""
    dev = _cuda_device(k_pages)
    num_pages, page_size, Hkv, d = pools = k_pages.shape
    B = block_table.shape[0]
    bt, max_blocks, sl = _table(block_table, seqlens, B, dev)
    _call("attn_kvcache_bounds_paged", dev, stream, _need("k_pages", k_pages, _BF16, pools, dev),
          _need("k_bounds", k_bounds, _BF16, (num_pages, page_size // 64, Hkv, 2, d), dev), bt, max_blocks, page_size,
          num_pages, sl, None if new_lens is None else _need("new_lens", new_lens, _I32, (B,), dev), B, max_new, Hkv, d)


def select_blocks_paged(q, k_bounds, block_table, seqlens, topk, sink=1, local=1, workspace=None, stream=None):
    """The topk blocks of 64 keys whose bounds allow the largest scores, for each of the last Nq tokens q [B,Nq,Hq,d]
    of each sequence (row i at position seqlens - Nq + i) and each KV head: int32 [B, Nq, Hkv, topk], ascending, -1 behind
    the last; the first `sink` and the last `local` blocks that a token sees are among them
    (attn_select_blocks_paged)."""
    dev = _cuda_device(q)
    if stream is not None:
        with _on(stream, dev):
            return select_blocks_paged(q, k_bounds, block_table, seqlens, topk, sink, local, workspace)
    B, Nq, Hq, d = q.shape
    shape = k_bounds.shape
    if len(shape) != 5 or shape[3:] != (2, d):
        raise ValueError("k_bounds must be [num_pages, page_size / 64, Hkv, 2, %d] (got %s)" % (d, tuple(shape)))
    num_pages, page_size, Hkv = shape[0], 64 * shape[1], shape[2]
    bt, max_blocks, sl = _table(block_table, seqlens, B, dev)
    args = (_need("q", q, _BF16, q.shape, dev), _need("k_bounds", k_bounds, _BF16, shape, dev), bt, max_blocks,
            page_size, num_pages, sl)
    blocks = torch.empty((B, Nq, Hkv, topk), dtype=_I32, device=dev)
    if workspace is None:
        n = _fn("attn_select_blocks_workspace_size")(B, Nq, Hkv, min(max_blocks * page_size, 0x7fffffff))
        workspace = torch.empty(n if n > 16 else 16, dtype=torch.uint8, device=dev)
    ws, n = _space(workspace, dev)
    _call("attn_select_blocks_paged", dev, None, *args, blocks.data_ptr(), B, Nq, Hq, Hkv, d, topk, sink, local, ws, n)
    return blocks


def attend_blocks_paged(q, k_pages, v_pages, block_table, seqlens, blocks, scale, workspace=None, stream=None):
    """Attention of each of the last Nq tokens q [B,Nq,Hq,d] bf16 of each sequence (row i at position seqlens - Nq + i)
    over the 64-key blocks listed for it and its KV head, blocks int32 [B, Nq, Hkv, n] (attn_fwd_blocks_paged).  Returns
    (o, lse [B,Hq,Nq])."""
    dev = _cuda_device(q)
    if stream is not None:
        with _on(stream, dev):
            return attend_blocks_paged(q, k_pages, v_pages, block_table, seqlens, blocks, scale, workspace)
    pools, Hkv = _pools(q, k_pages, v_pages, block_table, seqlens, dev)
    n_sel = blocks.shape[-1]
    return _attend("attn_fwd_blocks_paged", "attn_fwd_blocks_paged_workspace_size", q, pools, Hkv,
                   (_need("blocks", blocks, _I32, q.shape[:2] + (Hkv, n_sel), dev), n_sel), scale, workspace, dev,
                   n_sel, min(pools[4] * pools[5], 0x7fffffff))


def attn_get_device_status(stream=None):
    return lib().attn_get_device_status(_stream_handle(stream))


def attn_selftest_exp2_poly(x, y, stream=None):
    """y = 2^x by the library's software exp2 (float32 CUDA tensors of one size). Returns the status."""
    for name, t in (("x", x), ("y", y)):
        if t.dtype != torch.float32 or not t.is_cuda or not t.is_contiguous():
            raise ValueError("%s must be a contiguous CUDA float32 tensor" % name)
    if x.numel() != y.numel():
        raise ValueError("x and y differ in size")
    return lib().attn_selftest_exp2_poly(_ptr(x), _ptr(y), x.numel(), _stream_handle(stream))


def attn_probe_read_bandwidth(buf, sink, stream=None):
    """One streaming read of the CUDA tensor buf (its bytes; see the C call);
    sink: a CUDA int64 tensor of one element.  Returns the status."""
    if not buf.is_cuda or not buf.is_contiguous() or sink.dtype != torch.int64 or not sink.is_cuda:
        raise ValueError("buf must be a contiguous CUDA tensor and sink a CUDA int64 tensor")
    return lib().attn_probe_read_bandwidth(_ptr(buf), buf.numel() * buf.element_size(), _ptr(sink),
                                           _stream_handle(stream))


def attn_selftest_wait_timeout(limit_ns, stream=None):
    """Launches the bounded-wait self-test kernel; its timeout shows in attn_get_device_status."""
    return lib().attn_selftest_wait_timeout(int(limit_ns), _stream_handle(stream))


# --------------------------------------------------------------------------- convenience wrappers
def forward(q, k, v, causal, scale, stream=None, library=None):
    """Allocates O and LSE with torch on q's device and runs attn_fwd. Returns (o, lse)."""
    B, Nq, Hq, d = q.shape
    o = torch.empty_like(q)
    lse = torch.empty((B, Hq, Nq), dtype=torch.float32, device=q.device)
    rc = attn_fwd(q, k, v, o, lse, causal, scale, stream, library)
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_fwd")
    return o, lse


def forward_window(q, k, v, causal, window, scale, stream=None):
    """Allocates O and LSE and runs attn_fwd_window. Returns (o, lse)."""
    B, Nq, Hq, d = q.shape
    o = torch.empty_like(q)
    lse = torch.empty((B, Hq, Nq), dtype=torch.float32, device=q.device)
    rc = attn_fwd_window(q, k, v, o, lse, causal, window, scale, stream)
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_fwd_window")
    return o, lse


def decode_paged(q, k_pages, v_pages, block_table, seqlens, scale, chunk=1024, workspace=None, stream=None):
    """Allocates O, LSE (and the workspace unless given) and runs attn_fwd_splitkv_paged."""
    B, _, Hq, d = q.shape
    o = torch.empty_like(q)
    lse = torch.empty((B, Hq, 1), dtype=torch.float32, device=q.device)
    if workspace is None:
        n = attn_splitkv_workspace_size(B, Hq, block_table.shape[1] * k_pages.shape[1], d, chunk)
        workspace = torch.empty(max(n, 16), dtype=torch.uint8, device=q.device)
    rc = attn_fwd_splitkv_paged(q, k_pages, v_pages, block_table, seqlens, o, lse, scale, chunk, workspace, stream)
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_fwd_splitkv_paged")
    return o, lse


def decode(q, k_cache, v_cache, seqlens, scale, chunk=1024, workspace=None, stream=None):
    """Allocates O, LSE (and the workspace unless given) and runs attn_fwd_splitkv."""
    B, _, Hq, d = q.shape
    o = torch.empty_like(q)
    lse = torch.empty((B, Hq, 1), dtype=torch.float32, device=q.device)
    if workspace is None:
        n = attn_splitkv_workspace_size(B, Hq, k_cache.shape[1], d, chunk)
        workspace = torch.empty(max(n, 16), dtype=torch.uint8, device=q.device)
    rc = attn_fwd_splitkv(q, k_cache, v_cache, seqlens, o, lse, scale, chunk, workspace, stream)
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_fwd_splitkv")
    return o, lse

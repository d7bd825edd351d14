// Position rotation of one head row, shared by the norm-and-rotation and the
// cache-append kernels.
//
// A row of D values is held by D/16 neighbouring threads, two 16-byte chunks
// (8 bf16 each) a thread.  The first rot values are rotated in pairs, pair i
// by the angle whose cosine and sine the tables hold in entry i of the
// token's position: pairs (x_i, x_{i + rot/2}) (half-split) or (x_2i,
// x_{2i+1}) (interleaved).  A thread owns chunks l and l + rot/16 of the
// rotated part, so both values of a half-split pair sit in one thread and no
// exchange between threads is needed; threads beyond rot/16 own two
// neighbouring chunks of the rest.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "ptx.cuh"

namespace attn {

struct RopeParams {
  const float* cosv;  // [max_pos, rot / 2]
  const float* sinv;
  int max_pos, rot, inter;  // rot 0: no rotation (tables unused)
};

// The two chunks of thread l (of D/16) of a row.
__device__ __forceinline__ int2 row_chunks(int l, int rot) {
  const int half = rot >> 4;
  return l < half ? make_int2(l, l + half) : make_int2(2 * l, 2 * l + 1);
}

struct Angles {
  float c[8], s[8];
};

// Ordinary loads: these kernels start while earlier ones, which may write what
// is read here, still run, so nothing is constant over a kernel's time and no
// load may be moved before grid_depends.
__device__ __forceinline__ void load4(const float* p, float* r) {
  const float4 v = *reinterpret_cast<const float4*>(p);
  r[0] = v.x; r[1] = v.y; r[2] = v.z; r[3] = v.w;
}

// Cosines and sines of the 8 pairs of thread l at position pos (any l; those
// past the rotated part get the identity).  Half-split: pairs 8l .. 8l+7 of
// (chunk l, chunk l + rot/16).  Interleaved: pairs 4c .. 4c+3 of each chunk c.
__device__ __forceinline__ void load_angles(const RopeParams& rp, int pos, int l, Angles& a) {
  if (l >= (rp.rot >> 4)) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      a.c[i] = 1.f;
      a.s[i] = 0.f;
    }
    return;
  }
  const size_t row = static_cast<size_t>(pos) * (rp.rot >> 1);
  const int i0 = rp.inter ? 4 * l : 8 * l;
  const int i1 = rp.inter ? 4 * (l + (rp.rot >> 4)) : 8 * l + 4;
  load4(rp.cosv + row + i0, a.c);
  load4(rp.cosv + row + i1, a.c + 4);
  load4(rp.sinv + row + i0, a.s);
  load4(rp.sinv + row + i1, a.s + 4);
}

__device__ __forceinline__ void unpack8(const uint4& u, float* x) {
  x[0] = bf16lo(u.x); x[1] = bf16hi(u.x); x[2] = bf16lo(u.y); x[3] = bf16hi(u.y);
  x[4] = bf16lo(u.z); x[5] = bf16hi(u.z); x[6] = bf16lo(u.w); x[7] = bf16hi(u.w);
}
__device__ __forceinline__ uint4 pack8(const float* x) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}

// One pair, or two at once (packed products): each product and sum rounded by
// itself (no fused multiply-add), so the value that a cache's 8-bit code is
// taken from does not depend on the compiler's contraction.  kBack: by the
// negative angle (the transpose).  The sums of two pairs are not packed: packed
// products and sums were contracted in spite of their rounding modifiers.
template <bool kBack>
__device__ __forceinline__ void rotate_pair(float& a, float& b, float c, float s) {
  const float ac = __fmul_rn(a, c), bs = __fmul_rn(b, s), bc = __fmul_rn(b, c), as = __fmul_rn(a, s);
  a = kBack ? __fadd_rn(ac, bs) : __fsub_rn(ac, bs);
  b = kBack ? __fsub_rn(bc, as) : __fadd_rn(bc, as);
}
template <bool kBack>
__device__ __forceinline__ void rotate_two(float* a, float* b, const float* c, const float* s) {
  const float2 a2 = make_float2(a[0], a[1]), b2 = make_float2(b[0], b[1]), c2 = make_float2(c[0], c[1]),
               s2 = make_float2(s[0], s[1]);
  const float2 ac = fmul2(a2, c2), bs = fmul2(b2, s2), bc = fmul2(b2, c2), as = fmul2(a2, s2);
  a[0] = kBack ? __fadd_rn(ac.x, bs.x) : __fsub_rn(ac.x, bs.x);
  a[1] = kBack ? __fadd_rn(ac.y, bs.y) : __fsub_rn(ac.y, bs.y);
  b[0] = kBack ? __fsub_rn(bc.x, as.x) : __fadd_rn(bc.x, as.x);
  b[1] = kBack ? __fsub_rn(bc.y, as.y) : __fadd_rn(bc.y, as.y);
}

// Rotates a thread's 16 values x (chunk 0 in x[0..7], chunk 1 in x[8..15]).
template <bool kInter, bool kBack>
__device__ __forceinline__ void rotate16(float* x, const Angles& a) {
  if (kInter) {
#pragma unroll
    for (int i = 0; i < 8; ++i) rotate_pair<kBack>(x[2 * i], x[2 * i + 1], a.c[i], a.s[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; i += 2) rotate_two<kBack>(x + i, x + 8 + i, a.c + i, a.s + i);
  }
}

}  // namespace attn

// Softmax of one 128 x 128 score tile in Tensor Memory, a thread for each row
// (TMEM lane), as the attention over a paged bf16 cache uses it.  Scores are
// handled in base 2 and scaled: x = s c with c = scale log2(e) of either sign,
// p = 2^(x - M) under the row's exponent reference M, which is set by the
// row's first visible scores and moved only when a half's sum of p passes 2^16,
// so that p stays within what bf16 P and fp32 sums hold at full relative
// precision.  P replaces the scores, packed as bf16 pairs in the tile's first
// 64 columns; rounding p to bf16 is the tensor core's operand type, the sum of
// the weights takes p before it.
#pragma once
#include "ptx.cuh"

namespace attn {

// Visible columns of a tile's two halves of 64 for this row: the first v[h].
struct Visible {
  int v[2];
};

constexpr float kSumLimit = 65536.f;

__device__ __forceinline__ float rows_sum(float2 a0, float2 a1) { return (a0.x + a0.y) + (a1.x + a1.y); }

// p of 32 scores into 16 words of P.
__device__ __forceinline__ void rows_quarter(const uint32_t (&u)[32], float c, float M, float2& a0, float2& a1, uint32_t* pk) {
  const float2 c2 = make_float2(c, c), m2 = make_float2(-M, -M);
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float2 x = ffma2(make_float2(__uint_as_float(u[2 * i]), __uint_as_float(u[2 * i + 1])), c2, m2);
    const float2 e = make_float2(ex2_approx(x.x), ex2_approx(x.y));
    if (i & 1)
      a1 = fadd2(a1, e);
    else
      a0 = fadd2(a0, e);
    pk[i] = pack_bf16x2(e.x, e.y);
  }
}

// What a tile did to a row: its sum of p under the reference M that it leaves.
struct RowTile {
  float sum, M;
};

// Quarters q0 .. q1 - 1 of the tile in two passes.  First their largest visible
// score: it sets a reference that is not set, and moves it where it passes it by
// `over`.  Then P under the reference.  Rolled: this is the rare form, and the
// code of all warps has to stay in the instruction cache.
__device__ __forceinline__ RowTile rows_two_passes(uint32_t tS, int q0, int q1, const Visible& vis, float c, float M, float over) {
  float mt = -INFINITY;
#pragma unroll 1
  for (int q = q0; q < q1; ++q) {
    uint32_t u[32];
    tmem_ld32(tS + 32 * q, u);
    tmem_wait_ld();
    const int lim = (q < 2 ? vis.v[0] : vis.v[1]) - 32 * (q & 1);
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
      const float x0 = __uint_as_float(u[i]) * c, x1 = __uint_as_float(u[i + 1]) * c;
      mt = fmax3(mt, i < lim ? x0 : -INFINITY, i + 1 < lim ? x1 : -INFINITY);
    }
  }
  if (M == -INFINITY || mt - M > over) M = fmaxf(M, mt);
  const float m = M == -INFINITY ? 0.f : M;
  float sum = 0.f;
#pragma unroll 1
  for (int q = q0; q < q1; ++q) {
    uint32_t u[32], pk[16];
    tmem_ld32(tS + 32 * q, u);
    tmem_wait_ld();
    const int lim = (q < 2 ? vis.v[0] : vis.v[1]) - 32 * (q & 1);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float p0 = ex2_approx(fmaf(__uint_as_float(u[2 * i]), c, -m)), p1 = ex2_approx(fmaf(__uint_as_float(u[2 * i + 1]), c, -m));
      const float v0 = 2 * i < lim ? p0 : 0.f, v1 = 2 * i + 1 < lim ? p1 : 0.f;
      sum += v0 + v1;
      pk[i] = pack_bf16x2(v0, v1);
    }
    tmem_st16(tS + 16 * q, pk);
  }
  return {sum, M};
}

// Masked tiles, and those with the first scores of some row of the warp.
__device__ __noinline__ RowTile rows_first(uint32_t tS, Visible vis, float c, float M) {
  return rows_two_passes(tS, 0, 4, vis, c, M, 8.f);
}

// A half whose sum passed kSumLimit in some rows (ov), its scores still in
// place: those rows take its largest score as reference.  Second half: the first
// half's P (sum t0) lies in the tile under the old reference and is rescaled.
__device__ __noinline__ RowTile rows_fix(uint32_t tS, int half, float c, float M, float t0, bool ov) {
  const Visible all = {{64, 64}};
  const RowTile t = rows_two_passes(tS, 2 * half, 2 * half + 2, all, c, M, ov ? 0.f : INFINITY);
  if (half == 0) return t;
  const float f = ov ? ex2_approx(M - t.M) : 1.f;
  tmem_wait_st();
  uint32_t u[32];
  tmem_ld32(tS, u);
  tmem_wait_ld();
#pragma unroll
  for (int i = 0; i < 32; ++i) u[i] = f != 1.f ? pack_bf16x2(bf16lo(u[i]) * f, bf16hi(u[i]) * f) : u[i];
  tmem_st32(tS, u);
  return {t0 * f + t.sum, t.M};
}

// One pass over a tile whose columns are all seen, for warps whose live rows
// all have a reference.  Each quarter's scores are on their way while the one
// before is worked on.
__device__ __forceinline__ RowTile rows_tile(uint32_t tS, float c, float M, bool live) {
  float2 a0 = make_float2(0.f, 0.f), a1 = make_float2(0.f, 0.f);
  uint32_t ua[32], ub[32], pk[32];
  tmem_ld32(tS, ua);
  tmem_wait_ld();
  tmem_ld32(tS + 32, ub);
  rows_quarter(ua, c, M, a0, a1, pk);
  tmem_wait_ld();
  tmem_ld32(tS + 64, ua);
  rows_quarter(ub, c, M, a0, a1, pk + 16);
  tmem_wait_ld();
  float t0 = rows_sum(a0, a1);
  const bool ov0 = live && !(t0 <= kSumLimit);
  if (__any_sync(0xffffffffu, ov0)) {
    const RowTile f = rows_fix(tS, 0, c, M, 0.f, ov0);
    if (ov0) {
      M = f.M;
      t0 = f.sum;
      a0 = make_float2(t0, 0.f);
      a1 = make_float2(0.f, 0.f);
    }
  } else {
    tmem_st32(tS, pk);
  }
  tmem_ld32(tS + 96, ub);
  rows_quarter(ua, c, M, a0, a1, pk);
  tmem_wait_ld();
  rows_quarter(ub, c, M, a0, a1, pk + 16);
  float total = rows_sum(a0, a1);
  const bool ov1 = live && !(total - t0 <= kSumLimit);
  if (__any_sync(0xffffffffu, ov1)) {
    const RowTile f = rows_fix(tS, 1, c, M, t0, ov1);
    if (ov1) {
      M = f.M;
      total = f.sum;
    }
  } else {
    tmem_st32(tS + 32, pk);
  }
  return {total, M};
}

}  // namespace attn

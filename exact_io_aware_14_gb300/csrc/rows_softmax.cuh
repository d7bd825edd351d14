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

// p of 32-column quarter q into pairs (q & 1) * 16 .. of the half's packed P.
template <bool kMasked>
__device__ __forceinline__ void rows_quarter(const uint32_t (&u)[32], int q, const Visible& vis, float c, float M,
                                             float2& a0, float2& a1, uint32_t (&pk)[32]) {
  const float2 c2 = make_float2(c, c), m2 = make_float2(-M, -M);
  const int lim = kMasked ? vis.v[q >> 1] - 32 * (q & 1) : 32;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float2 x = ffma2(make_float2(__uint_as_float(u[2 * i]), __uint_as_float(u[2 * i + 1])), c2, m2);
    float p0 = ex2_approx(x.x), p1 = ex2_approx(x.y);
    if (kMasked) {
      p0 = 2 * i < lim ? p0 : 0.f;
      p1 = 2 * i + 1 < lim ? p1 : 0.f;
    }
    if (i & 1)
      a1 = fadd2(a1, make_float2(p0, p1));
    else
      a0 = fadd2(a0, make_float2(p0, p1));
    pk[(q & 1) * 16 + i] = pack_bf16x2(p0, p1);
  }
}

__device__ __forceinline__ float rows_sum(float2 a0, float2 a1) { return (a0.x + a0.y) + (a1.x + a1.y); }

// Largest scaled score of half h, -inf if none is visible.
template <bool kMasked>
__device__ __forceinline__ float rows_half_max(uint32_t tS, int h, const Visible& vis, float c) {
  float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    uint32_t u[32];
    tmem_ld32(tS + 64 * h + 32 * k, u);
    tmem_wait_ld();
    const int lim = kMasked ? vis.v[h] - 32 * k : 32;
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
      float x0 = __uint_as_float(u[i]) * c, x1 = __uint_as_float(u[i + 1]) * c;
      if (kMasked) {
        x0 = i < lim ? x0 : -INFINITY;
        x1 = i + 1 < lim ? x1 : -INFINITY;
      }
      if (i & 2)
        m1 = fmax3(m1, x0, x1);
      else
        m0 = fmax3(m0, x0, x1);
    }
  }
  return fmaxf(m0, m1);
}

// Half h under reference M, stored.  Returns its sum.
template <bool kMasked>
__device__ __forceinline__ float rows_half(uint32_t tS, int h, const Visible& vis, float c, float M) {
  float2 a0 = make_float2(0.f, 0.f), a1 = make_float2(0.f, 0.f);
  uint32_t u[32], pk[32];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    tmem_ld32(tS + 64 * h + 32 * k, u);
    tmem_wait_ld();
    rows_quarter<kMasked>(u, 2 * h + k, vis, c, M, a0, a1, pk);
  }
  tmem_st32(tS + 32 * h, pk);
  return rows_sum(a0, a1);
}

// What a tile did to a row: its sum of p under the reference M that it leaves.
struct RowTile {
  float sum, M;
};

// First visible scores of some row of the warp: the tile's largest score sets
// a reference that is not set, or moves one that it passes by 2^8.
template <bool kMasked>
__device__ __noinline__ RowTile rows_first(uint32_t tS, Visible vis, float c, float M) {
  const float mt = fmaxf(rows_half_max<kMasked>(tS, 0, vis, c), rows_half_max<kMasked>(tS, 1, vis, c));
  if (M == -INFINITY || mt - M > 8.f) M = fmaxf(M, mt);
  const float m = M == -INFINITY ? 0.f : M;
  float sum = rows_half<kMasked>(tS, 0, vis, c, m);
  sum += rows_half<kMasked>(tS, 1, vis, c, m);
  return {sum, M};
}

// A half whose sum passed kSumLimit in some rows (ov), its scores still in
// place: those rows take its largest score as reference.  kSecond: the first
// half's P (sum t0) lies in the tile under the old reference and is rescaled.
template <bool kMasked, bool kSecond>
__device__ __noinline__ RowTile rows_fix(uint32_t tS, Visible vis, float c, float M, float t0, bool ov) {
  const float mx = rows_half_max<kMasked>(tS, kSecond ? 1 : 0, vis, c);
  float f = 1.f;
  if (ov) {
    const float m_new = fmaxf(M, mx);
    f = ex2_approx(M - m_new);
    M = m_new;
  }
  const float sum = rows_half<kMasked>(tS, kSecond ? 1 : 0, vis, c, M);
  if (!kSecond) return {sum, M};
  tmem_wait_st();
  uint32_t u[32];
  tmem_ld32(tS, u);
  tmem_wait_ld();
#pragma unroll
  for (int i = 0; i < 32; ++i) u[i] = f != 1.f ? pack_bf16x2(bf16lo(u[i]) * f, bf16hi(u[i]) * f) : u[i];
  tmem_st32(tS, u);
  return {t0 * f + sum, M};
}

// One pass over the tile, for warps whose live rows all have a reference.  Each
// quarter's scores are on their way while the one before is worked on.
template <bool kMasked>
__device__ __forceinline__ RowTile rows_tile(uint32_t tS, const Visible& vis, float c, float M, bool live) {
  float2 a0 = make_float2(0.f, 0.f), a1 = make_float2(0.f, 0.f);
  uint32_t ua[32], ub[32], pk[32];
  tmem_ld32(tS, ua);
  tmem_wait_ld();
  tmem_ld32(tS + 32, ub);
  rows_quarter<kMasked>(ua, 0, vis, c, M, a0, a1, pk);
  tmem_wait_ld();
  tmem_ld32(tS + 64, ua);
  rows_quarter<kMasked>(ub, 1, vis, c, M, a0, a1, pk);
  tmem_wait_ld();
  float t0 = rows_sum(a0, a1);
  const bool ov0 = live && !(t0 <= kSumLimit);
  if (__any_sync(0xffffffffu, ov0)) {
    const RowTile f = rows_fix<kMasked, false>(tS, vis, c, M, 0.f, ov0);
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
  rows_quarter<kMasked>(ua, 2, vis, c, M, a0, a1, pk);
  tmem_wait_ld();
  rows_quarter<kMasked>(ub, 3, vis, c, M, a0, a1, pk);
  float total = rows_sum(a0, a1);
  const bool ov1 = live && !(total - t0 <= kSumLimit);
  if (__any_sync(0xffffffffu, ov1)) {
    const RowTile f = rows_fix<kMasked, true>(tS, vis, c, M, t0, ov1);
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

// Joining the pieces of a row of attention over a paged bf16 cache: each is a
// normalised output and its log-sum-exp (base 2) in fp32,
//     LSE = log2 sum 2^LSE_i,  O = sum 2^(LSE_i - LSE) O_i,
// in order.  A warp a row.
#pragma once
#include <cuda_bf16.h>

#include "launch.h"
#include "ptx.cuh"

namespace attn {
namespace {

constexpr int kJoinWarps = 4;

struct Join {
  float m, l;
};
// A row's pieces, `count` of them: `place(i)` is the row of piece i in the
// workspace, -1 where there is none.  32 at a time, a lane a piece for the
// weights; the outputs are on their way meanwhile.
template <int D, typename Params, typename Place>
__device__ __forceinline__ void join(const Params& p, int count, Place place, Join& s, float (&acc)[D / 32]) {
  constexpr int kV = D / 32;
  const int lane = threadIdx.x & 31;
  for (int i0 = 0; i0 < count; i0 += 32) {
    const int n = min(32, count - i0);
    const long long at = lane < n ? place(i0 + lane) : -1;
    const uint32_t have = __ballot_sync(0xffffffffu, at >= 0);
    const float mine = at >= 0 ? p.lse_part[at] : -INFINITY;
    float m = mine;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    m = fmaxf(m, s.m);
    const float ref = m == -INFINITY ? 0.f : m;
    const float a = ex2_approx(s.m - ref);  // 0 while nothing was seen
    const float w = mine != mine ? mine : ex2_approx(mine - ref);
    s.m = m;
    s.l *= a;
#pragma unroll
    for (int x = 0; x < kV; ++x) acc[x] *= a;
    for (int i = 0; i < n; i += 8) {
      float v[8][kV];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float* o = p.o_part + __shfl_sync(0xffffffffu, at, (i + k) & 31) * D + lane * kV;
        if (have >> ((i + k) & 31) & 1u) {
          if constexpr (kV == 4)
            *reinterpret_cast<float4*>(v[k]) = *reinterpret_cast<const float4*>(o);
          else
            *reinterpret_cast<float2*>(v[k]) = *reinterpret_cast<const float2*>(o);
        }
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float wi = __shfl_sync(0xffffffffu, w, (i + k) & 31);
        if (have >> ((i + k) & 31) & 1u) {
          s.l += wi;
#pragma unroll
          for (int x = 0; x < kV; ++x) acc[x] = fmaf(wi, v[k][x], acc[x]);
        }
      }
    }
  }
}

template <int D, typename Params>
__device__ __forceinline__ void write_row(const Params& p, int tok, int hq, const Join& s, const float (&acc)[D / 32]) {
  const int lane = threadIdx.x & 31;
  const float inv = s.l == 0.f ? 0.f : 1.f / s.l;
  uint32_t* o = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.o) + (static_cast<long long>(tok) * p.Hq + hq) * D +
                                            lane * (D / 32));
#pragma unroll
  for (int x = 0; x < D / 64; ++x) o[x] = pack_bf16x2(acc[2 * x] * inv, acc[2 * x + 1] * inv);
  if (lane == 0) {
    const int b = tok / p.Nq;
    p.lse[(static_cast<long long>(b) * p.Hq + hq) * p.Nq + tok - b * p.Nq] =
        s.l == 0.f ? -INFINITY : (s.m + __log2f(s.l)) * 0.6931471805599453f;
  }
}

}  // namespace
}  // namespace attn

// Attention of query rows over a paged bf16 cache, for sm_103a: over a whole
// sequence (whose first keys the batch may share), or over listed 64-key blocks.
//
// One CTA for a row and head: 64 keys at a time, two threads a score, a
// running maximum m and sum l, each thread one or two output channels.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "launch.h"
#include "ptx.cuh"
#include "rope.cuh"

namespace attn {
namespace {

__device__ uint32_t g_rows_status;

__device__ __forceinline__ void record(uint32_t site, uint32_t code) {
  atomicCAS(&g_rows_status, 0u, (site << 8) | code);
}

template <int D>
__global__ void __launch_bounds__(128) rows_kernel(const RowsParams p) {
  __shared__ float s_q[D], s_p[64], s_m[4];
  const int tid = threadIdx.x;
  const int hq = blockIdx.x % p.Hq, token = blockIdx.x / p.Hq;
  const int b = token / p.Nq, n = token % p.Nq;
  const int hkv = hq / (p.Hq / p.Hkv);
  const int cap = p.max_blocks * p.page_size;
  int len = p.seqlens[b];
  if (tid == 0 && hq == 0 && n == 0 && (len < 0 || len > cap)) record(1, kDevBadSeqlen);
  len = min(max(len, 0), cap);
  const int seen = max(0, len - p.Nq + n + 1);
  if (tid < D) s_q[tid] = __bfloat162float(static_cast<const __nv_bfloat16*>(p.q)[(static_cast<long long>(token) * p.Hq + hq) * D + tid]);
  float m = -INFINITY, l = 0.f, acc = 0.f;
  const int steps = p.blocks ? p.n_sel : (seen + 63) / 64;
  for (int s = 0; s < steps; ++s) {
    int blk = s;
    if (p.blocks) {
      blk = p.blocks[(static_cast<long long>(token) * p.Hkv + hkv) * p.n_sel + s];
      if (blk >= cap / 64 && tid == 0) record(2, kDevBadPage);
      if (blk < 0 || blk >= cap / 64 || blk * 64 >= seen) continue;
    }
    const int v = min(64, seen - blk * 64);
    const int row = blk * 64 < p.shared_len ? 0 : b;
    int pg = p.block_table[static_cast<long long>(row) * p.max_blocks + blk * 64 / p.page_size];
    if (pg < 0 || pg >= p.num_pages) {
      if (tid == 0) record(3, kDevBadPage);
      pg = 0;
    }
    const long long at = ((static_cast<long long>(pg) * p.page_size + blk * 64 % p.page_size) * p.Hkv + hkv) * D;
    const int key = tid >> 1, half = tid & 1;
    float x = 0.f;
    __syncthreads();
    if (key < v) {
      const __nv_bfloat16* k = static_cast<const __nv_bfloat16*>(p.k_pages) + at + static_cast<long long>(key) * p.Hkv * D + half * (D / 2);
      for (int i = 0; i < D / 2; i += 8) {
        float f[8];
        unpack8(*reinterpret_cast<const uint4*>(k + i), f);
        for (int j = 0; j < 8; ++j) x = fmaf(f[j], s_q[half * (D / 2) + i + j], x);
      }
    }
    x += __shfl_xor_sync(0xffffffffu, x, 1);
    x = key < v ? x * p.scale_log2 : -INFINITY;
    float mx = x;
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    if ((tid & 31) == 0) s_m[tid >> 5] = mx;
    __syncthreads();
    const float mn = fmaxf(fmaxf(fmaxf(s_m[0], s_m[1]), fmaxf(s_m[2], s_m[3])), m);
    if (half == 0) s_p[key] = key < v ? ex2_approx(x - mn) : 0.f;
    __syncthreads();
    const float a = m == -INFINITY ? 0.f : ex2_approx(m - mn);
    m = mn;
    float sum = 0.f, pv = 0.f;
    for (int j = 0; j < v; ++j) {
      sum += s_p[j];
      if (tid < D) pv = fmaf(s_p[j], __bfloat162float(static_cast<const __nv_bfloat16*>(p.v_pages)[at + static_cast<long long>(j) * p.Hkv * D + tid]), pv);
    }
    l = l * a + sum;
    acc = acc * a + pv;
  }
  if (tid < D)
    static_cast<__nv_bfloat16*>(p.o)[(static_cast<long long>(token) * p.Hq + hq) * D + tid] = __float2bfloat16(l == 0.f ? 0.f : acc / l);
  if (tid == 0)
    p.lse[(static_cast<long long>(b) * p.Hq + hq) * p.Nq + n] = l == 0.f ? -INFINITY : (m + __log2f(l)) * 0.6931471805599453f;
}

}  // namespace

cudaError_t launch_rows(const RowsParams& p, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>(p.B * p.Nq * p.Hq);
  if (p.d == 64)
    rows_kernel<64><<<grid, 128, 0, stream>>>(p);
  else
    rows_kernel<128><<<grid, 128, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t status_word_rows(uint32_t** at) { return cudaGetSymbolAddress(reinterpret_cast<void**>(at), g_rows_status); }

}  // namespace attn

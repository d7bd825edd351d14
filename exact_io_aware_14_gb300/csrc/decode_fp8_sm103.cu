// Split-KV decode of one or a few new tokens over a paged e4m3 cache with one
// scale for each page and KV head, for sm_103a.
//
//   s_j = scale * ks[page(j)] * <q, kc_j>,  o = sum_j p_j vs[page(j)] vc_j / sum_j p_j
//
// Simple form: one block per (row, split of the keys, sequence), a thread a
// key for the scores and a thread a dim for the output.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "launch.h"
#include "ptx.cuh"

namespace attn {
namespace {

__device__ uint32_t g_decode_fp8_status;

__device__ __forceinline__ void record(uint32_t site, uint32_t code) {
  atomicCAS(&g_decode_fp8_status, 0u, (site << 8) | code);
}

__device__ __forceinline__ float2 from_e4m3x2(uint16_t u) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(u));
  float lo, hi;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(lo), "=f"(hi)
      : "r"(h));
  return make_float2(lo, hi);
}

constexpr int kTile = 128;

template <int D>
__global__ void __launch_bounds__(kTile) decode_fp8_simple_kernel(const DecodeFp8Params p) {
  __shared__ float s_q[D], s_p[kTile], s_red[4];
  __shared__ int s_page[kTile];
  const int tid = threadIdx.x;
  const int hq = blockIdx.x % p.Hq, i = blockIdx.x / p.Hq;
  const int b = blockIdx.y, split = blockIdx.z;
  const int hkv = hq / (p.Hq / p.Hkv);
  int Lb = p.seqlens[b];
  if (Lb < 0 || Lb > p.max_seqlen) {
    if (tid == 0) record(1, kDevBadSeqlen);
    Lb = Lb < 0 ? 0 : p.max_seqlen;
  }
  const int k0 = split * p.chunk;
  if (k0 >= Lb) return;
  const int lim = min(Lb - p.Nq + i + 1, k0 + p.chunk);  // keys [k0, lim)
  const long long qrow = (static_cast<long long>(b) * p.Nq + i) * p.Hq + hq;
  if (tid < D) s_q[tid] = __bfloat162float(static_cast<const __nv_bfloat16*>(p.q)[qrow * D + tid]);
  float m = -INFINITY, l = 0.f, acc = 0.f;
  for (int t0 = k0; t0 < lim; t0 += kTile) {
    __syncthreads();
    const int key = t0 + tid;
    float s = -INFINITY, vs = 0.f;
    int pg = 0;
    if (key < lim) {
      pg = p.block_table[static_cast<long long>(b) * p.max_blocks + key / p.page_size];
      if (pg < 0 || pg >= p.num_pages) {
        record(2, kDevBadPage);
        pg = 0;
      }
      const uint16_t* k = reinterpret_cast<const uint16_t*>(
          static_cast<const uint8_t*>(p.k_pages) +
          ((static_cast<long long>(pg) * p.page_size + key % p.page_size) * p.Hkv + hkv) * D);
      float dot = 0.f;
      for (int c = 0; c < D / 2; ++c) {
        const float2 kv = from_e4m3x2(k[c]);
        dot = fmaf(s_q[2 * c], kv.x, dot);
        dot = fmaf(s_q[2 * c + 1], kv.y, dot);
      }
      s = dot * p.k_scales[static_cast<long long>(pg) * p.Hkv + hkv] * p.scale_log2;
      vs = p.v_scales[static_cast<long long>(pg) * p.Hkv + hkv];
    }
    float mt = s;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, o));
    if ((tid & 31) == 0) s_red[tid >> 5] = mt;
    __syncthreads();
    mt = fmaxf(fmaxf(s_red[0], s_red[1]), fmaxf(s_red[2], s_red[3]));
    const float m_new = fmaxf(m, mt);
    const float alpha = m == -INFINITY ? 0.f : exp2f(m - m_new);
    const float pr = (key < lim) ? exp2f(s - m_new) : 0.f;
    m = m_new;
    float sum = pr;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    __syncthreads();
    if ((tid & 31) == 0) s_red[tid >> 5] = sum;
    s_p[tid] = pr * vs;
    s_page[tid] = pg;
    __syncthreads();
    l = l * alpha + (s_red[0] + s_red[1]) + (s_red[2] + s_red[3]);
    if (tid < D) {
      acc *= alpha;
      for (int j = 0; j < kTile && t0 + j < lim; ++j) {
        const uint16_t code = static_cast<const uint8_t*>(
            p.v_pages)[((static_cast<long long>(s_page[j]) * p.page_size + (t0 + j) % p.page_size) * p.Hkv + hkv) * D + tid];
        acc = fmaf(s_p[j], from_e4m3x2(code).x, acc);
      }
    }
  }
  const long long row = qrow * p.n_split + split;
  if (tid < D) p.o_part[row * D + tid] = l == 0.f ? 0.f : acc / l;
  // l is 0 exactly where the row sees no key of the split (NaN, not 0, where a score is NaN)
  if (tid == 0) p.lse_part[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

// One block per row of q: LSE = ln sum_s exp(LSE_s), O = sum_s exp(LSE_s - LSE) O_s.
template <int D>
__global__ void __launch_bounds__(D) decode_fp8_combine_kernel(const DecodeFp8Params p) {
  const long long qrow = blockIdx.x;
  const int hq = static_cast<int>(qrow % p.Hq);
  const int i = static_cast<int>(qrow / p.Hq % p.Nq);
  const int b = static_cast<int>(qrow / p.Hq / p.Nq);
  const int dd = threadIdx.x;
  int Lb = p.seqlens[b];
  Lb = Lb < 0 ? 0 : (Lb > p.max_seqlen ? p.max_seqlen : Lb);
  const int ns = (Lb + p.chunk - 1) / p.chunk;
  const float* lp = p.lse_part + qrow * p.n_split;
  const float* op = p.o_part + qrow * p.n_split * D + dd;
  float mx = -INFINITY;
  for (int s = 0; s < ns; ++s) mx = fmaxf(mx, lp[s]);
  if (mx == -INFINITY) mx = 0.f;  // no key seen (or every LSE NaN): the weights are then 0 (NaN)
  float tot = 0.f, acc = 0.f;
  for (int s = 0; s < ns; ++s) {
    const float w = expf(lp[s] - mx);
    tot += w;
    acc = fmaf(w, op[static_cast<long long>(s) * D], acc);
  }
  const bool none = tot == 0.f;
  static_cast<__nv_bfloat16*>(p.o)[qrow * D + dd] = __float2bfloat16_rn(none ? 0.f : acc / tot);
  if (dd == 0) p.lse[(static_cast<long long>(b) * p.Hq + hq) * p.Nq + i] = none ? -INFINITY : mx + logf(tot);
}

template <int D>
cudaError_t launch_d(const DecodeFp8Params& p, cudaStream_t stream) {
  decode_fp8_simple_kernel<D><<<dim3(p.Nq * p.Hq, p.B, p.n_split), kTile, 0, stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  decode_fp8_combine_kernel<D><<<static_cast<unsigned>(p.B) * p.Nq * p.Hq, D, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_decode_fp8(const DecodeFp8Params& p, cudaStream_t stream) {
  return p.d == 64 ? launch_d<64>(p, stream) : launch_d<128>(p, stream);
}

cudaError_t fetch_status_decode_fp8(cudaStream_t stream, uint32_t* out) {
  uint32_t zero = 0;
  cudaError_t e =
      cudaMemcpyFromSymbolAsync(out, g_decode_fp8_status, sizeof(uint32_t), 0, cudaMemcpyDeviceToHost, stream);
  if (e == cudaSuccess)
    e = cudaMemcpyToSymbolAsync(g_decode_fp8_status, &zero, sizeof(uint32_t), 0, cudaMemcpyHostToDevice, stream);
  if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
  return e;
}

}  // namespace attn

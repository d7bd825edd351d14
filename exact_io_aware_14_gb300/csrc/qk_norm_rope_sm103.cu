// Norms of queries and keys for each head with the position rotation in the
// same pass, forward and backward, for sm_103a.
//
//   forward   y = R(x * r * w),  r = 1 / sqrt(mean(x^2) + eps)
//   backward  u = R^T dy,  g = u * w,  xr = x * r
//             dx = r * (g - xr * mean(g * xr)),  dw = sum over rows of u * xr
// Without a weight there is no norm: y = R(x), dx = R^T dy.
//
// Both are bound by memory (about 4 flops a byte), so each value is read and
// written once, 16 bytes a thread and access: D/16 threads hold a row, two
// chunks each (rope.cuh), the mean square is a shuffle reduction over them,
// and the rotation needs no exchange.  A group of threads takes kHeads heads
// of one token, whose loads are all issued before the first is used and
// which share the token's cosines and sines.
//
// The backward pass needs x again to recompute r, so the forward pass saves
// nothing.  dw: every thread keeps its 16 columns' sums in 32 bits over the
// rows it walks, the block adds them in a fixed order into one row of the
// workspace, and a second kernel adds those rows in a fixed order (no
// atomics: the same inputs give the same bits).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "launch.h"
#include "ptx.cuh"
#include "rope.cuh"

namespace attn {
namespace {

__device__ uint32_t g_rope_status;

constexpr int kThreads = 256;

__device__ __forceinline__ int checked_pos(int pos, int max_pos) {
  if (pos < 0 || pos >= max_pos) {
    atomicCAS(&g_rope_status, 0u, (1u << 8) | static_cast<uint32_t>(kDevBadPosition));
    return pos < 0 ? 0 : max_pos - 1;
  }
  return pos;
}

template <int kTPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = kTPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// One work item: up to kHeads heads of one token, q's or k's.
struct Item {
  bool is_k;
  int h0, nh;        // first head, heads (0: no item)
  long long token;   // b * N + n
};
template <int kHeads>
__device__ __forceinline__ Item item_of(long long i, long long n_items, int gq, int gk, int Hq, int Hkv) {
  Item it;
  const int per = gq + gk;
  it.token = i / per;
  const int g = static_cast<int>(i - it.token * per);
  it.is_k = g >= gq;
  it.h0 = (it.is_k ? g - gq : g) * kHeads;
  it.nh = i < n_items ? min(kHeads, (it.is_k ? Hkv : Hq) - it.h0) : 0;
  return it;
}

template <int D, int kHeads, bool kInter>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_kernel(const QkNormRopeParams p, long long n_items, int gq,
                                                               int gk) {
  constexpr int kTPR = D / 16;
  const int l = threadIdx.x % kTPR;
  const long long i = (static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x) / kTPR;
  const Item it = item_of<kHeads>(i, n_items, gq, gk, p.Hq, p.Hkv);  // nh 0 past the end: no load or store
  const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(it.is_k ? p.k : p.q) +
                           it.token * (it.is_k ? p.k_stride : p.q_stride) + static_cast<long long>(it.h0) * D;
  const int2 ch = row_chunks(l, p.rope.rot);
  uint4 raw[kHeads][2];
#pragma unroll
  for (int h = 0; h < kHeads; ++h) {
    raw[h][0] = raw[h][1] = make_uint4(0u, 0u, 0u, 0u);
    if (h < it.nh) {
      raw[h][0] = *reinterpret_cast<const uint4*>(x + h * D + 8 * ch.x);
      raw[h][1] = *reinterpret_cast<const uint4*>(x + h * D + 8 * ch.y);
    }
  }
  Angles ang;
  const bool turn = p.rope.rot > 0 && it.nh > 0;
  if (turn) {
    const int pos = p.positions ? p.positions[it.token] : static_cast<int>(it.token % p.N);
    load_angles(p.rope, checked_pos(pos, p.rope.max_pos), l, ang);
  }
  const float* w = it.is_k ? p.k_weight : p.q_weight;
  float wv[16];
  if (w) {
    load4(w + 8 * ch.x, wv);
    load4(w + 8 * ch.x + 4, wv + 4);
    load4(w + 8 * ch.y, wv + 8);
    load4(w + 8 * ch.y + 4, wv + 12);
  }
  __nv_bfloat16* y = static_cast<__nv_bfloat16*>(it.is_k ? p.k_out : p.q_out) +
                     (it.token * (it.is_k ? p.Hkv : p.Hq) + it.h0) * D;
#pragma unroll
  for (int h = 0; h < kHeads; ++h) {
    float v[16];
    unpack8(raw[h][0], v);
    unpack8(raw[h][1], v + 8);
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < 16; ++j) ss = fmaf(v[j], v[j], ss);
    ss = row_sum<kTPR>(ss);
    if (w) {
      const float r = rsqrtf(fmaf(ss, 1.f / D, p.eps));
#pragma unroll
      for (int j = 0; j < 16; ++j) v[j] = v[j] * r * wv[j];
    }
    if (turn && l < (p.rope.rot >> 4)) rotate16<kInter, false>(v, ang);
    if (h < it.nh) {
      *reinterpret_cast<uint4*>(y + h * D + 8 * ch.x) = pack8(v);
      *reinterpret_cast<uint4*>(y + h * D + 8 * ch.y) = pack8(v + 8);
    }
  }
}

// Backward.  Blocks [0, nbq) walk q's items, the rest k's, each a fixed set,
// so a block's dw row belongs to one of the two weights.
template <int D, int kHeads, bool kInter>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_bwd_kernel(const QkNormRopeParams p, int nbq, int nbk) {
  constexpr int kTPR = D / 16;
  constexpr int kGroups = kThreads / kTPR;
  const bool is_k = static_cast<int>(blockIdx.x) >= nbq;
  const int nb = is_k ? nbk : nbq, blk = is_k ? blockIdx.x - nbq : blockIdx.x;
  const int H = is_k ? p.Hkv : p.Hq, per = (H + kHeads - 1) / kHeads;
  const long long n_items = static_cast<long long>(p.B) * p.N * per;
  const __nv_bfloat16* x0 = static_cast<const __nv_bfloat16*>(is_k ? p.k : p.q);
  const long long stride = is_k ? p.k_stride : p.q_stride;
  const __nv_bfloat16* dy0 = static_cast<const __nv_bfloat16*>(is_k ? p.dk_out : p.dq_out);
  __nv_bfloat16* dx0 = static_cast<__nv_bfloat16*>(is_k ? p.dk : p.dq);
  const float* w = is_k ? p.k_weight : p.q_weight;
  const int l = threadIdx.x % kTPR;
  const int2 ch = row_chunks(l, p.rope.rot);
  float wv[16], dw[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) dw[j] = 0.f;
  if (w) {
    load4(w + 8 * ch.x, wv);
    load4(w + 8 * ch.x + 4, wv + 4);
    load4(w + 8 * ch.y, wv + 8);
    load4(w + 8 * ch.y + 4, wv + 12);
  }
  // every group of a warp makes the same number of rounds: the row sums are warp-wide shuffles
  const long long step = static_cast<long long>(nb) * kGroups;
  for (long long base = static_cast<long long>(blk) * kGroups; base < n_items; base += step) {
    const long long i = base + threadIdx.x / kTPR;
    const long long token = i / per;
    const int h0 = static_cast<int>(i - token * per) * kHeads;
    const int nh = i < n_items ? min(kHeads, H - h0) : 0;
    const __nv_bfloat16* x = x0 + token * stride + static_cast<long long>(h0) * D;
    const long long dense = (token * H + h0) * D;
    uint4 rx[kHeads][2], rd[kHeads][2];
#pragma unroll
    for (int h = 0; h < kHeads; ++h) {
      rx[h][0] = rx[h][1] = rd[h][0] = rd[h][1] = make_uint4(0u, 0u, 0u, 0u);
      if (h < nh) {
        rd[h][0] = *reinterpret_cast<const uint4*>(dy0 + dense + h * D + 8 * ch.x);
        rd[h][1] = *reinterpret_cast<const uint4*>(dy0 + dense + h * D + 8 * ch.y);
        if (w) {
          rx[h][0] = *reinterpret_cast<const uint4*>(x + h * D + 8 * ch.x);
          rx[h][1] = *reinterpret_cast<const uint4*>(x + h * D + 8 * ch.y);
        }
      }
    }
    Angles ang;
    const bool turn = p.rope.rot > 0 && nh > 0;
    if (turn) {
      const int pos = p.positions ? p.positions[token] : static_cast<int>(token % p.N);
      load_angles(p.rope, checked_pos(pos, p.rope.max_pos), l, ang);
    }
#pragma unroll
    for (int h = 0; h < kHeads; ++h) {
      float u[16], v[16];
      unpack8(rd[h][0], u);
      unpack8(rd[h][1], u + 8);
      if (turn && l < (p.rope.rot >> 4)) rotate16<kInter, true>(u, ang);
      if (w) {  // uniform over the block
        unpack8(rx[h][0], v);
        unpack8(rx[h][1], v + 8);
        float ss = 0.f, gx = 0.f;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          ss = fmaf(v[j], v[j], ss);
          gx = fmaf(u[j] * wv[j], v[j], gx);
        }
        ss = row_sum<kTPR>(ss);
        gx = row_sum<kTPR>(gx);
        const float r = rsqrtf(fmaf(ss, 1.f / D, p.eps));
        const float m = gx * r * (1.f / D);  // mean(g * xr)
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const float xr = v[j] * r;
          dw[j] = fmaf(u[j], xr, dw[j]);
          u[j] = r * fmaf(-xr, m, u[j] * wv[j]);
        }
      }
      if (h < nh) {
        *reinterpret_cast<uint4*>(dx0 + dense + h * D + 8 * ch.x) = pack8(u);
        *reinterpret_cast<uint4*>(dx0 + dense + h * D + 8 * ch.y) = pack8(u + 8);
      }
    }
  }
  if (!w) return;
  __shared__ float s_dw[kThreads / 32][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
#pragma unroll
    for (int o = kTPR; o < 32; o <<= 1) dw[j] += __shfl_xor_sync(0xffffffffu, dw[j], o);
    if (lane < kTPR) s_dw[warp][8 * (j < 8 ? ch.x : ch.y) + (j & 7)] = dw[j];
  }
  __syncthreads();
  for (int c = threadIdx.x; c < D; c += kThreads) {
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < kThreads / 32; ++k) s += s_dw[k][c];
    p.dw_part[static_cast<size_t>(blockIdx.x) * D + c] = s;
  }
}

// Adds the blocks' dw rows: block 0 q's, block 1 k's; 1024/D threads a
// column, then a fixed-order sum over them.
template <int D>
__global__ void __launch_bounds__(1024) qk_norm_rope_dw_kernel(const float* part, int nbq, int nbk, float* dwq,
                                                               float* dwk) {
  constexpr int kPer = 1024 / D;
  float* out = blockIdx.x == 0 ? dwq : dwk;
  if (!out) return;
  __shared__ float s_sum[kPer][D];
  const int c = threadIdx.x % D, g = threadIdx.x / D;
  const int lo = blockIdx.x == 0 ? 0 : nbq, n = blockIdx.x == 0 ? nbq : nbk;
  float s = 0.f;
  for (int i = g; i < n; i += kPer) s += part[static_cast<size_t>(lo + i) * D + c];
  s_sum[g][c] = s;
  __syncthreads();
  if (g == 0) {
#pragma unroll
    for (int k = 1; k < kPer; ++k) s += s_sum[k][c];
    out[c] = s;
  }
}

template <int D, int kHeads>
cudaError_t launch_fwd(const QkNormRopeParams& p, cudaStream_t stream) {
  const int gq = (p.Hq + kHeads - 1) / kHeads, gk = (p.Hkv + kHeads - 1) / kHeads;
  const long long items = static_cast<long long>(p.B) * p.N * (gq + gk);
  const unsigned blocks = static_cast<unsigned>((items * (D / 16) + kThreads - 1) / kThreads);
  if (p.rope.inter)
    qk_norm_rope_kernel<D, kHeads, true><<<blocks, kThreads, 0, stream>>>(p, items, gq, gk);
  else
    qk_norm_rope_kernel<D, kHeads, false><<<blocks, kThreads, 0, stream>>>(p, items, gq, gk);
  return cudaGetLastError();
}

constexpr int kBwdHeads = 2;

template <int D>
cudaError_t launch_bwd(const QkNormRopeParams& p, int nbq, int nbk, cudaStream_t stream) {
  if (p.rope.inter)
    qk_norm_rope_bwd_kernel<D, kBwdHeads, true><<<nbq + nbk, kThreads, 0, stream>>>(p, nbq, nbk);
  else
    qk_norm_rope_bwd_kernel<D, kBwdHeads, false><<<nbq + nbk, kThreads, 0, stream>>>(p, nbq, nbk);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || (!p.dq_weight && !p.dk_weight)) return e;
  qk_norm_rope_dw_kernel<D><<<2, 1024, 0, stream>>>(p.dw_part, nbq, nbk, p.dq_weight, p.dk_weight);
  return cudaGetLastError();
}

}  // namespace

void qk_norm_rope_bwd_blocks(int B, int N, int Hq, int Hkv, int d, int* nbq, int* nbk) {
  // blocks for about the rows there are, at most kMax in all, shared out by heads
  constexpr int kMax = 152 * 6;
  const long long groups = kThreads / (d / 16);
  const long long tokens = static_cast<long long>(B) * N;
  auto want = [&](int H, int cap) {
    const long long n = (tokens * ((H + kBwdHeads - 1) / kBwdHeads) + groups - 1) / groups;
    return static_cast<int>(n < 1 ? 1 : (n > cap ? cap : n));
  };
  int cap_q = static_cast<int>(static_cast<long long>(kMax) * Hq / (Hq + Hkv));
  cap_q = cap_q < 1 ? 1 : (cap_q > kMax - 1 ? kMax - 1 : cap_q);
  *nbq = want(Hq, cap_q);
  *nbk = Hkv > 0 ? want(Hkv, kMax - cap_q) : 0;
}

cudaError_t launch_qk_norm_rope(const QkNormRopeParams& p, cudaStream_t stream) {
  if (p.d == 64) return launch_fwd<64, 4>(p, stream);
  return launch_fwd<128, 4>(p, stream);
}

cudaError_t launch_qk_norm_rope_bwd(const QkNormRopeParams& p, cudaStream_t stream) {
  int nbq, nbk;
  qk_norm_rope_bwd_blocks(p.B, p.N, p.Hq, p.Hkv, p.d, &nbq, &nbk);
  if (p.d == 64) return launch_bwd<64>(p, nbq, nbk, stream);
  return launch_bwd<128>(p, nbq, nbk, stream);
}

cudaError_t fetch_status_rope(cudaStream_t stream, uint32_t* out) {
  uint32_t zero = 0;
  cudaError_t e = cudaMemcpyFromSymbolAsync(out, g_rope_status, sizeof(uint32_t), 0, cudaMemcpyDeviceToHost, stream);
  if (e == cudaSuccess)
    e = cudaMemcpyToSymbolAsync(g_rope_status, &zero, sizeof(uint32_t), 0, cudaMemcpyHostToDevice, stream);
  if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
  return e;
}

}  // namespace attn

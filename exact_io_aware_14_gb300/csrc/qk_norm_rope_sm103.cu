// Norms of queries and keys for each head with the position rotation in the
// same pass, forward and backward, for sm_103a.
//
//   forward   y = R(x * r * w),  r = 1 / sqrt(mean(x^2) + eps)
//   backward  u = R^T dy,  g = u * w,  xr = x * r
//             dx = r * (g - xr * mean(g * xr)),  dw = sum over rows of u * xr
// Without a weight there is no norm: y = R(x), dx = R^T dy.
//
// Both are bound by memory (about 4 flops a byte), so each value is read and
// written once: D/16 threads hold a row, two 16-byte chunks each (rope.cuh),
// the mean square is a shuffle reduction over them, and the rotation needs no
// exchange.
//
// Two forms, chosen by size (launch rules below):
//   short   (forward) a group of threads takes one row of one token: the
//           least latency
//   long    a fixed grid of CTAs walks q's items and k's (kHeads heads of one
//           token, which share its cosines and sines).  As soon as a head's
//           values are unpacked, its registers take the same head of the
//           group's next item, so loads stay in flight while the arithmetic
//           runs
// Tiles brought into shared memory by bulk copies were slower (105 us on the
// training forward against 61.5 for plain loads into registers without the
// overlap): a row's angles are then read again for each head, and the
// instructions, twice as many, became the limit.
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

// The short form: row i of the q and k rows of all tokens (a token's q heads,
// then its k heads).
template <int D, bool kInter>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_kernel(const QkNormRopeParams p, long long rows) {
  grid_depends();
  constexpr int kTPR = D / 16;
  const int l = threadIdx.x % kTPR;
  const long long i = (static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x) / kTPR;
  const bool has = i < rows;  // the others take part in the shuffles
  const int per = p.Hq + p.Hkv;
  const long long token = i / per;
  int h = static_cast<int>(i - token * per);
  const bool is_k = h >= p.Hq;
  if (is_k) h -= p.Hq;
  const int2 ch = row_chunks(l, p.rope.rot);
  float v[16];
  uint4 raw[2];
  raw[0] = raw[1] = make_uint4(0u, 0u, 0u, 0u);
  if (has) {
    const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(is_k ? p.k : p.q) +
                             token * (is_k ? p.k_stride : p.q_stride) + static_cast<long long>(h) * D;
    raw[0] = *reinterpret_cast<const uint4*>(x + 8 * ch.x);
    raw[1] = *reinterpret_cast<const uint4*>(x + 8 * ch.y);
  }
  Angles ang;
  const bool turn = has && l < (p.rope.rot >> 4);
  if (turn) {
    const int pos = p.positions ? p.positions[token] : static_cast<int>(token % p.N);
    load_angles(p.rope, checked_pos(pos, p.rope.max_pos), l, ang);
  }
  const float* w = is_k ? p.k_weight : p.q_weight;
  float wv[16];
  if (w) {
    load4(w + 8 * ch.x, wv);
    load4(w + 8 * ch.x + 4, wv + 4);
    load4(w + 8 * ch.y, wv + 8);
    load4(w + 8 * ch.y + 4, wv + 12);
  }
  unpack8(raw[0], v);
  unpack8(raw[1], v + 8);
  float ss = 0.f;
#pragma unroll
  for (int j = 0; j < 16; ++j) ss = fmaf(v[j], v[j], ss);
  ss = row_sum<kTPR>(ss);
  if (w) {
    const float r = rsqrtf(fmaf(ss, 1.f / D, p.eps));
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] = v[j] * r * wv[j];
  }
  if (turn) rotate16<kInter, false>(v, ang);
  if (has) {
    __nv_bfloat16* y = static_cast<__nv_bfloat16*>(is_k ? p.k_out : p.q_out) +
                       (token * (is_k ? p.Hkv : p.Hq) + h) * D;
    *reinterpret_cast<uint4*>(y + 8 * ch.x) = pack8(v);
    *reinterpret_cast<uint4*>(y + 8 * ch.y) = pack8(v + 8);
  }
}

// ---------------------------------------------------------------------------
// The long form.

// How one of the two tensors is shared out.
struct RowPlan {
  int H, blocks;
  FastDiv per;  // items of a token
};
struct LongPlan {
  RowPlan q, k;
  FastDiv by_N;
};

// kStream: the tensors do not fit L2, whose lines loads and stores then give up first.
template <int D, int kHeads, int kMinBlocks, bool kInter, bool kBwd, bool kStream>
__global__ void __launch_bounds__(kThreads, kMinBlocks)
    qk_norm_rope_long_kernel(const QkNormRopeParams p, const LongPlan plan) {
  grid_depends();
  constexpr int kTPR = D / 16;
  constexpr int kGroups = kThreads / kTPR;
  const bool is_k = static_cast<int>(blockIdx.x) >= plan.q.blocks;
  const int H = is_k ? plan.k.H : plan.q.H;
  FastDiv per;
  per.d = is_k ? plan.k.per.d : plan.q.per.d;
  per.m = is_k ? plan.k.per.m : plan.q.per.m;
  per.s = is_k ? plan.k.per.s : plan.q.per.s;
  const unsigned step = (is_k ? plan.k.blocks : plan.q.blocks) * kGroups;
  const unsigned n_items = static_cast<unsigned>(p.B) * p.N * per.d;  // fits: checked on the host
  const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(is_k ? p.k : p.q);
  const long long stride = is_k ? p.k_stride : p.q_stride;
  const __nv_bfloat16* dy = static_cast<const __nv_bfloat16*>(is_k ? p.dk_out : p.dq_out);
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(kBwd ? (is_k ? p.dk : p.dq) : (is_k ? p.k_out : p.q_out));
  const float* w = is_k ? p.k_weight : p.q_weight;
  const bool need_x = !kBwd || w != nullptr;
  const int l = threadIdx.x % kTPR;
  const int2 ch = row_chunks(l, p.rope.rot);
  const bool turn = l < (p.rope.rot >> 4);  // this thread's chunks are rotated
  float wv[16], dw[kBwd ? 16 : 1];
  if (kBwd) {
#pragma unroll
    for (int j = 0; j < 16; ++j) dw[kBwd ? j : 0] = 0.f;
  }
  if (w) {
    load4(w + 8 * ch.x, wv);
    load4(w + 8 * ch.x + 4, wv + 4);
    load4(w + 8 * ch.y, wv + 8);
    load4(w + 8 * ch.y + 4, wv + 12);
  }

  // an item's place; nh 0 past the last
  struct Place {
    unsigned token;
    int h0, nh;
  };
  auto place = [&](unsigned i) {
    Place a;
    a.token = per.div(i);
    a.h0 = static_cast<int>(i - a.token * per.d) * kHeads;
    a.nh = i < n_items ? min(kHeads, H - a.h0) : 0;
    return a;
  };
  auto load16 = [](const __nv_bfloat16* at) {
    return kStream ? __ldcs(reinterpret_cast<const uint4*>(at)) : *reinterpret_cast<const uint4*>(at);
  };
  auto store16 = [](__nv_bfloat16* at, const uint4& v) {
    if (kStream)
      __stcs(reinterpret_cast<uint4*>(at), v);
    else
      *reinterpret_cast<uint4*>(at) = v;
  };
  uint4 rx[kHeads][2], rd[kBwd ? kHeads : 1][2];
  auto load_head = [&](const Place& a, int h) {
    rx[h][0] = rx[h][1] = make_uint4(0u, 0u, 0u, 0u);
    if (kBwd) rd[kBwd ? h : 0][0] = rd[kBwd ? h : 0][1] = make_uint4(0u, 0u, 0u, 0u);
    if (h < a.nh) {
      if (need_x) {
        const __nv_bfloat16* r = x + a.token * stride + static_cast<long long>(a.h0 + h) * D;
        rx[h][0] = load16(r + 8 * ch.x);
        rx[h][1] = load16(r + 8 * ch.y);
      }
      if (kBwd) {
        const __nv_bfloat16* r = dy + (static_cast<long long>(a.token) * H + a.h0 + h) * D;
        rd[kBwd ? h : 0][0] = load16(r + 8 * ch.x);
        rd[kBwd ? h : 0][1] = load16(r + 8 * ch.y);
      }
    }
  };
  auto position = [&](const Place& a) {
    if (p.rope.rot == 0 || a.nh == 0) return 0;
    return p.positions ? p.positions[a.token]
                       : static_cast<int>(a.token - plan.by_N.div(a.token) * plan.by_N.d);
  };
  auto angles = [&](const Place& a, int pos, Angles& ang) {
    if (turn && a.nh > 0) load_angles(p.rope, checked_pos(pos, p.rope.max_pos), l, ang);
  };

  // every group of a warp makes the same number of rounds: the row sums are warp-wide shuffles
  const unsigned first = (is_k ? blockIdx.x - plan.q.blocks : blockIdx.x) * kGroups;
  const unsigned grp = threadIdx.x / kTPR;
  Place cur = place(first + grp);
  Angles ang;
#pragma unroll
  for (int h = 0; h < kHeads; ++h) load_head(cur, h);
  angles(cur, position(cur), ang);
  Place nxt = place(first + step + grp);
  int pos_nxt = position(nxt);
  for (unsigned base = first; base < n_items; base += step) {
    const Place after = place(base + 2 * step + grp);
    const int pos_after = position(after);
#pragma unroll
    for (int h = 0; h < kHeads; ++h) {
      float y[16], v[kBwd ? 16 : 1];
      if (!kBwd) {
        unpack8(rx[h][0], y);
        unpack8(rx[h][1], y + 8);
      } else {
        unpack8(rd[kBwd ? h : 0][0], y);
        unpack8(rd[kBwd ? h : 0][1], y + 8);
        unpack8(rx[h][0], v);
        unpack8(rx[h][1], v + (kBwd ? 8 : 0));
      }
      load_head(nxt, h);
      if (!kBwd) {
        if (w) {
          float ss = 0.f;
#pragma unroll
          for (int j = 0; j < 16; ++j) ss = fmaf(y[j], y[j], ss);
          ss = row_sum<kTPR>(ss);
          const float rs = rsqrtf(fmaf(ss, 1.f / D, p.eps));
#pragma unroll
          for (int j = 0; j < 16; ++j) y[j] = y[j] * rs * wv[j];
        }
        if (turn) rotate16<kInter, false>(y, ang);
        if (h == kHeads - 1) angles(nxt, pos_nxt, ang);
      } else {
        if (turn) rotate16<kInter, true>(y, ang);
        if (h == kHeads - 1) angles(nxt, pos_nxt, ang);
        if (w) {
          float ss = 0.f, gx = 0.f;
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float vj = v[kBwd ? j : 0];
            ss = fmaf(vj, vj, ss);
            gx = fmaf(y[j] * wv[j], vj, gx);
          }
          ss = row_sum<kTPR>(ss);
          gx = row_sum<kTPR>(gx);
          const float rs = rsqrtf(fmaf(ss, 1.f / D, p.eps));
          const float m = gx * rs * (1.f / D);  // mean(g * xr)
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float xr = v[kBwd ? j : 0] * rs;
            if (h < cur.nh) dw[kBwd ? j : 0] = fmaf(y[j], xr, dw[kBwd ? j : 0]);
            y[j] = rs * fmaf(-xr, m, y[j] * wv[j]);
          }
        }
      }
      if (h < cur.nh) {
        __nv_bfloat16* o = out + (static_cast<long long>(cur.token) * H + cur.h0 + h) * D;
        store16(o + 8 * ch.x, pack8(y));
        store16(o + 8 * ch.y, pack8(y + 8));
      }
    }
    cur = nxt;
    nxt = after;
    pos_nxt = pos_after;
  }
  if (!kBwd || !w) return;
  __shared__ float s_dw[kBwd ? kThreads / 32 : 1][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    float v = dw[kBwd ? j : 0];
#pragma unroll
    for (int o = kTPR; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (lane < kTPR) s_dw[kBwd ? warp : 0][8 * (j < 8 ? ch.x : ch.y) + (j & 7)] = v;
  }
  __syncthreads();
  if (threadIdx.x < D) {
    float v = 0.f;
#pragma unroll
    for (int k = 0; k < kThreads / 32; ++k) v += s_dw[kBwd ? k : 0][threadIdx.x];
    p.dw_part[static_cast<size_t>(blockIdx.x) * D + threadIdx.x] = v;
  }
}

// Adds the blocks' dw rows, 32 columns of one tensor a block: 32 warps take
// every 32nd row (loads independent of one another), then their sums are
// added in a fixed order.
template <int D>
__global__ void __launch_bounds__(1024) qk_norm_rope_dw_kernel(const float* part, int nbq, int nbk, float* dwq,
                                                               float* dwk) {
  grid_depends();
  const bool is_k = blockIdx.x >= D / 32;
  float* out = is_k ? dwk : dwq;
  if (!out) return;
  __shared__ float s_sum[32][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c = blockIdx.x % (D / 32) * 32 + lane;
  const int lo = is_k ? nbq : 0, n = is_k ? nbk : nbq;
  float s = 0.f;
#pragma unroll 8
  for (int i = warp; i < n; i += 32) s += part[static_cast<size_t>(lo + i) * D + c];
  s_sum[warp][lane] = s;
  __syncthreads();
  if (warp == 0) {
#pragma unroll
    for (int k = 1; k < 32; ++k) s += s_sum[k][lane];
    out[c] = s;
  }
}

// Launch rules, each with both sides measured (GB300, d = 128 where not said).
// Long forward from 2 M values on: 1.0 M (32 + 8 heads) short 3.0 us, long
// 3.2; 4.1 M 5.8 and 4.3; 33 M 35 and 25.
constexpr long long kLongElements = 1 << 21;
// Heads of an item: four where that leaves few places empty (33 M values, 32
// + 8 heads: four 25.1 us, two 25.5, one 29.5), else one (12 M, 5 + 1 heads, d
// = 64: 18.6, 13.5 and 11.8).  Two CTAs of 128 registers a thread: with three
// the loads in flight spill (119 us for 58).  Backward: two heads (88 us; one
// 135, four with one CTA 100).
constexpr int kBwdHeads = 2, kCtasPerSm = 2;
int fwd_heads(int Hq, int Hkv) {
  const int places = (Hq + 3) / 4 * 4 + (Hkv + 3) / 4 * 4;
  return places * 10 <= (Hq + Hkv) * 11 ? 4 : 1;
}

// CTAs for q and for k by their share of the rows, no more than there is work for.
LongPlan plan_long(int B, int N, int Hq, int Hkv, int d, int heads) {
  LongPlan plan;
  const int ctas = 152 * kCtasPerSm;
  const int groups = kThreads / (d / 16);
  auto share = [&](int H, int cap) {
    RowPlan r;
    r.H = H;
    const int per = H == 0 ? 1 : (H + heads - 1) / heads;
    r.per = FastDiv(per);
    const long long want = (static_cast<long long>(B) * N * per + groups - 1) / groups;
    r.blocks = H == 0 ? 0 : static_cast<int>(want < 1 ? 1 : (want > cap ? cap : want));
    return r;
  };
  int nq = static_cast<int>(static_cast<long long>(ctas) * Hq / (Hq + Hkv));
  nq = nq < 1 ? 1 : (Hkv > 0 && nq > ctas - 1 ? ctas - 1 : nq);
  plan.q = share(Hq, nq);
  plan.k = share(Hkv, Hkv > 0 ? ctas - nq : 0);
  plan.by_N = FastDiv(N < 1 ? 1 : N);
  return plan;
}

template <int D, int kHeads, bool kInter, bool kBwd>
cudaError_t launch_long(const QkNormRopeParams& p, cudaStream_t stream) {
  const LongPlan plan = plan_long(p.B, p.N, p.Hq, p.Hkv, p.d, kHeads);
  // tensors past L2's 129 MB together (172 MB in, 172 MB out: 56.2 us streamed, 58.1 not)
  const bool past_l2 = static_cast<double>(p.B) * p.N * (p.Hq + p.Hkv) * D * 2 * (kBwd ? 3 : 2) > 129e6;
  const dim3 grid(plan.q.blocks + plan.k.blocks);
  cudaError_t e =
      past_l2 ? launch_dependent(qk_norm_rope_long_kernel<D, kHeads, kCtasPerSm, kInter, kBwd, true>, grid, kThreads, 0,
                                 stream, p, plan)
              : launch_dependent(qk_norm_rope_long_kernel<D, kHeads, kCtasPerSm, kInter, kBwd, false>, grid, kThreads, 0,
                                 stream, p, plan);
  if (!kBwd || e != cudaSuccess || (!p.dq_weight && !p.dk_weight)) return e;
  return launch_dependent(qk_norm_rope_dw_kernel<D>, dim3(2 * (D / 32)), 1024, 0, stream, p.dw_part, plan.q.blocks,
                          plan.k.blocks, p.dq_weight, p.dk_weight);
}

template <int D, bool kInter>
cudaError_t launch_fwd(const QkNormRopeParams& p, cudaStream_t stream) {
  const long long rows = static_cast<long long>(p.B) * p.N * (p.Hq + p.Hkv);
  if (rows * D >= kLongElements)
    return fwd_heads(p.Hq, p.Hkv) == 4 ? launch_long<D, 4, kInter, false>(p, stream)
                                       : launch_long<D, 1, kInter, false>(p, stream);
  const unsigned blocks = static_cast<unsigned>((rows * (D / 16) + kThreads - 1) / kThreads);
  return launch_dependent(qk_norm_rope_kernel<D, kInter>, dim3(blocks), kThreads, 0, stream, p, rows);
}

}  // namespace

void qk_norm_rope_bwd_blocks(int B, int N, int Hq, int Hkv, int d, int* nbq, int* nbk) {
  const LongPlan plan = plan_long(B, N, Hq, Hkv, d, kBwdHeads);
  *nbq = plan.q.blocks;
  *nbk = plan.k.blocks;
}

cudaError_t launch_qk_norm_rope(const QkNormRopeParams& p, cudaStream_t stream) {
  if (p.d == 64) return p.rope.inter ? launch_fwd<64, true>(p, stream) : launch_fwd<64, false>(p, stream);
  return p.rope.inter ? launch_fwd<128, true>(p, stream) : launch_fwd<128, false>(p, stream);
}

cudaError_t launch_qk_norm_rope_bwd(const QkNormRopeParams& p, cudaStream_t stream) {
  constexpr int h = kBwdHeads;
  if (p.d == 64)
    return p.rope.inter ? launch_long<64, h, true, true>(p, stream) : launch_long<64, h, false, true>(p, stream);
  return p.rope.inter ? launch_long<128, h, true, true>(p, stream) : launch_long<128, h, false, true>(p, stream);
}

cudaError_t status_word_rope(uint32_t** at) { return cudaGetSymbolAddress(reinterpret_cast<void**>(at), g_rope_status); }

}  // namespace attn

// Split-KV decode of one or a few new tokens over a paged e4m3 cache with one
// scale for each page and KV head, for sm_103a.
//
//   s_j = scale * ks[page(j)] * <q, kc_j>,  o = sum_j p_j vs[page(j)] vc_j / sum_j p_j
//
// The step is bound by reading the cache (2 d bytes a key and KV head).  At
// HBM speed that is about 23 codes a cycle and SM: converting them and
// multiplying them by 4 to 16 query rows on the CUDA cores would not keep
// up, so the codes go from memory through TMA into tcgen05 MMAs as they are,
// and no thread touches them:
//   S   [128 keys x N]  = K [128 x d]   Q^T        (A: the K tile, K-major)
//   O^T [d x N]         = V^T [d x 128] P^T        (A: the V tile, M-major)
// kind::f8f6f4 multiplies e4m3 by e5m2, so q and p are split into three e5m2
// terms each (3 significant bits a term: 9 bits, more than bf16's 8, and a
// range of 2^31 below the row's largest value): with R rows the MMA has N =
// 3R columns, the three terms of a row are added up in fp32 afterwards.
// q is scaled by a power of two a row (largest value in [2^14, 2^15)).  The
// weights p are formed with a running reference (moved only when a score
// passes it by 2^4) and multiplied by the page's value scale over the split's
// largest, times 2^10: at most 2^14, and what is lost is under 2^-27 of the
// largest value for each key.
//
// One CTA (10 warps) works on up to R query rows (heads of one KV head's
// group, times new tokens) of one sequence and one split of the keys:
//   warps 0-3  softmax, a thread a key (TMEM lane): scales, running
//              reference, weights, their three terms as bytes into shared
//              memory
//   warps 4-7  output, a thread a dim: adds each tile's O^T columns to its
//              fp32 registers (so no rescaling in TMEM)
//   warp 8     TMA loads, 128 keys of K and V a stage, in boxes of 64 rows
//              (pages are multiples of 64 rows)
//   warp 9     TMEM, MMA issue: S of tile t+1 goes out before O of tile t
// Two tiles of S, P and O are in flight, two CTAs fit an SM.
//
// Combine kernel: LSE = ln sum_s exp(LSE_s), O = sum_s exp(LSE_s - LSE) O_s.
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

constexpr int kTile = 128;     // keys per tile (MMA M of S, K of O^T)
constexpr int kThreads = 320;
constexpr uint64_t kWaitLimitNs = 2000000000ull;
constexpr float kMoveLog2 = 4.f;      // the reference moves when a score passes it by this
constexpr float kWeightScale = 1024.f;  // 2^10: weights up to 2^14, e5m2 ends at 57344

template <int D, int R>
struct Cfg {
  static constexpr int kN = (3 * R + 15) / 16 * 16;  // MMA columns
  static constexpr int kTmem = kN <= 16 ? 64 : (kN <= 32 ? 128 : 256);  // 4 kN, a power of two
  static constexpr int kCtas = R == 16 ? 1 : 2;                         // per SM (registers)
  static constexpr int kTileBytes = kTile * D;
  static constexpr int kStages = (R == 16 ? 6 : 3) * 128 / D;
  static constexpr int kOffV = 0;  // V first: the M-major reads of a 64-dim V tile run into K's (see below)
  static constexpr int kOffK = kTileBytes;
  static constexpr int kStage = 2 * kTileBytes;
  static constexpr int kOffQ = kStages * kStage;
  static constexpr int kOffP = kOffQ + (kN * D + 1023) / 1024 * 1024;  // [2][kN][128] bytes
  static constexpr int kOffScale = kOffP + 2 * kN * kTile;             // float ks, vs, int page [kMaxBlocks]
  static constexpr int kMaxBlocks = 256;                               // 64-key blocks of a split
  static constexpr int kOffAlpha = kOffScale + 3 * kMaxBlocks * 4;     // float [2][R]
  static constexpr int kOffRed = kOffAlpha + 2 * R * 4;                // float [4][R], then 4 flags
  static constexpr int kOffQm = kOffRed + 4 * R * 4 + 16;              // float qmul[R], m[R], l[4][R]
  static constexpr int kOffBar = (kOffQm + 6 * R * 4 + 15) / 16 * 16;  // full, empty [kStages], s, p, o, ofree [2]
  static constexpr int kNumBars = 2 * kStages + 9;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kBytes = kOffMisc + 16;
  static constexpr int kAlloc = kBytes + 1024;
};

__device__ __forceinline__ bool wait_all(uint64_t* bar, uint32_t parity, volatile int* abort_flag, uint32_t site) {
  bool ok = mbar_wait(bar, parity, abort_flag, kWaitLimitNs);
  ok = __all_sync(0xffffffffu, ok);
  if (!ok && (threadIdx.x & 31) == 0) record(site, kDevTimeout);
  return ok;
}
__device__ __forceinline__ bool wait_one(uint64_t* bar, uint32_t parity, volatile int* abort_flag, uint32_t site) {
  const bool ok = mbar_wait(bar, parity, abort_flag, kWaitLimitNs);
  if (!ok) record(site, kDevTimeout);
  return ok;
}

// named barrier 1 over the softmax warps, with an OR of a flag
__device__ __forceinline__ bool softmax_bar_or(bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred pi, po;\n\t"
      "setp.ne.u32 pi, %1, 0;\n\t"
      "bar.red.or.pred po, 1, 128, pi;\n\t"
      "selp.u32 %0, 1, 0, po;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(v))
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void softmax_bar() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

// two floats -> two e5m2 codes, `lo` in the low byte
__device__ __forceinline__ uint32_t e5m2x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// x cut to its 3 leading significant bits (what one e5m2 term holds)
__device__ __forceinline__ float lead3(float x) { return __uint_as_float(__float_as_uint(x) & 0xffe00000u); }

__device__ __forceinline__ void st_shared_u8(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.u8 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Byte offset of row n, byte c of an operand with rows of D bytes, swizzled
// as TMA and the MMA descriptors have it.
template <int kRow>
__device__ __forceinline__ int swizzled(int n, int c) {
  const int chunk = (c >> 4) ^ (kRow == 128 ? (n & 7) : ((n >> 1) & 3));
  return n * kRow + (chunk << 4) + (c & 15);
}

template <int kN>
__device__ __forceinline__ void tmem_ld_row(uint32_t addr, uint32_t (&u)[kN]) {
#pragma unroll
  for (int c = 0; c < kN; c += 16) tmem_ld16(addr + c, u + c);
  tmem_wait_ld();
}

template <int D, int R>
__global__ void __launch_bounds__(kThreads, Cfg<D, R>::kCtas) decode_fp8_split_kernel(const __grid_constant__ DecodeFp8Params p) {
  using C = Cfg<D, R>;
  constexpr int kN = C::kN;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  // grid (KV head x row block, sequence, split), high splits first: only long
  // sequences have them, and every low split is full
  const int G = p.Hq / p.Hkv;
  const int rows = p.Nq * G;  // query rows of a KV head: row r is token r / G, head r % G of the group
  const int n_rblk = (rows + R - 1) / R;
  const int hkv = blockIdx.x / n_rblk;
  const int row0 = (blockIdx.x % n_rblk) * R;
  const int nr = min(R, rows - row0);
  const int b = blockIdx.y, split = p.n_split - 1 - blockIdx.z;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  int Lb = p.seqlens[b];
  if (Lb < 0 || Lb > p.max_seqlen) {
    if (tid == 0 && blockIdx.x == 0) record(1, kDevBadSeqlen);
    Lb = Lb < 0 ? 0 : p.max_seqlen;
  }
  const int k0 = split * p.chunk;
  if (k0 >= Lb && !(p.n_split == 1)) return;  // empty split: the combine never reads it
  const int kn = max(0, min(p.chunk, Lb - k0));
  const int n_t = (kn + kTile - 1) / kTile;
  const int n_blk = (kn + 63) / 64;
  // keys of this split that row r sees: those below lim(r)
  auto lim = [&](int r) { return min(kn, Lb - p.Nq + (row0 + r) / G + 1 - k0); };
  const int lim_min = lim(0);

  float* s_ks = reinterpret_cast<float*>(smem + C::kOffScale);
  float* s_vs = s_ks + C::kMaxBlocks;
  int* s_page = reinterpret_cast<int*>(s_vs + C::kMaxBlocks);
  float* s_alpha = reinterpret_cast<float*>(smem + C::kOffAlpha);
  float* s_red = reinterpret_cast<float*>(smem + C::kOffRed);
  int* s_fail = reinterpret_cast<int*>(smem + C::kOffRed + 4 * R * 4);
  float* s_qm = reinterpret_cast<float*>(smem + C::kOffQm);
  float* s_m = s_qm + R;
  float* s_l = s_m + R;
  uint64_t* bar_full = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t* bar_empty = bar_full + C::kStages;
  uint64_t* bar_s = bar_empty + C::kStages;  // [2] S of a tile in TMEM
  uint64_t* bar_p = bar_s + 2;               // [2] P of a tile in shared memory (4 softmax warps)
  uint64_t* bar_o = bar_p + 2;               // [2] O^T of a tile in TMEM
  uint64_t* bar_of = bar_o + 2;              // [2] O^T and alpha read (D / 32 output warps)
  uint64_t* bar_drain = bar_of + 2;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
  const uint32_t sQ = smem_u32(smem + C::kOffQ), sP = smem_u32(smem + C::kOffP);

  int n_issued = 0;  // the loader's
  auto issue = [&](int t) {
    const int s = t % C::kStages;
    const int nb = min(2, n_blk - 2 * t);
    mbar_arrive_expect_tx(bar_full + s, 2 * nb * 64 * D);
    for (int i = 0; i < nb; ++i) {
      const int blk = 2 * t + i;
      const int row = (k0 + 64 * blk) % p.page_size, page = s_page[blk];
      tma_load_4d(smem + s * C::kStage + C::kOffK + i * 64 * D, &p.tm_k, bar_full + s, 0, hkv, row, page);
      tma_load_4d(smem + s * C::kStage + C::kOffV + i * 64 * D, &p.tm_v, bar_full + s, 0, hkv, row, page);
    }
  };

  if (warp == 8) {
    // barriers, the split's pages, and the first loads
    if (lane == 0) {
      for (int s = 0; s < C::kStages; ++s) {
        mbar_init(bar_full + s, 1);
        mbar_init(bar_empty + s, 1);
      }
      for (int i = 0; i < 2; ++i) {
        mbar_init(bar_s + i, 1);
        mbar_init(bar_p + i, 4);
        mbar_init(bar_o + i, 1);
        mbar_init(bar_of + i, D / 32);
      }
      mbar_init(bar_drain, 1);
      *abort_flag = 0;
      mbar_fence_init();
      tma_prefetch_desc(&p.tm_k);
      tma_prefetch_desc(&p.tm_v);
    }
    for (int i = lane; i < n_blk; i += 32) {
      int pg = p.block_table[static_cast<long long>(b) * p.max_blocks + (k0 + 64 * i) / p.page_size];
      if (pg < 0 || pg >= p.num_pages) {
        record(2, kDevBadPage);
        pg = 0;  // keep every load inside the page pool; the result is flagged
      }
      s_page[i] = pg;
    }
    __syncwarp();
    if (lane == 0) {
      for (int t = 0; t < n_t && t < C::kStages; ++t) issue(t);
      n_issued = min(n_t, C::kStages);
    }
  } else if (warp == 9) {
    tmem_alloc(s_tmem, C::kTmem);
    tmem_relinquish();
  } else if (warp < 4) {
    // scales of the split's 64-key blocks
    for (int i = tid; i < n_blk; i += 128) {
      int pg = p.block_table[static_cast<long long>(b) * p.max_blocks + (k0 + 64 * i) / p.page_size];
      if (pg < 0 || pg >= p.num_pages) pg = 0;
      s_ks[i] = p.k_scales[static_cast<long long>(pg) * p.Hkv + hkv];
      s_vs[i] = p.v_scales[static_cast<long long>(pg) * p.Hkv + hkv];
    }
  } else {
    // q as three e5m2 terms a row: column term * R + r
    const int w4 = warp - 4;
    for (int r = w4; r < R; r += 4) {
      float x[D / 32];
      float amax = 0.f;
      bool fin = true;
      const int tok = (row0 + r) / G, hq = hkv * G + (row0 + r) % G;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        x[i] = 0.f;
        if (r < nr)
          x[i] = __bfloat162float(static_cast<const __nv_bfloat16*>(
              p.q)[((static_cast<long long>(b) * p.Nq + tok) * p.Hq + hq) * D + (D / 32) * lane + i]);
        fin = fin && fabsf(x[i]) < INFINITY;
        amax = fmaxf(amax, fabsf(x[i]));
      }
      amax = warp_max(amax);
      fin = __all_sync(0xffffffffu, fin);
      const int e = fin ? max(static_cast<int>(__float_as_uint(amax) >> 23) - 127, -100) : 0;
      const float f = __uint_as_float(static_cast<uint32_t>(14 - e + 127) << 23);
      uint32_t term[3] = {0u, 0u, 0u};
#pragma unroll
      for (int i = 0; i < D / 32; i += 2) {
        float a = fin ? x[i] * f : 0.f, c = fin ? x[i + 1] * f : 0.f;
#pragma unroll
        for (int k = 0; k < 3; ++k) {
          const float ta = lead3(a), tc = lead3(c);
          term[k] |= e5m2x2(ta, tc) << (8 * i);
          a -= ta;
          c -= tc;
        }
      }
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        const uint32_t at = sQ + swizzled<D>(k * R + r, (D / 32) * lane);
        if (D == 128)
          asm volatile("st.shared.u32 [%0], %1;" ::"r"(at), "r"(term[k]) : "memory");
        else
          asm volatile("st.shared.u16 [%0], %1;" ::"r"(at), "h"(static_cast<uint16_t>(term[k])) : "memory");
      }
      // a row with an infinity or NaN: every score NaN
      if (lane == 0)
        s_qm[r] = fin ? __uint_as_float(static_cast<uint32_t>(e - 14 + 127) << 23) * p.scale_log2 : NAN;
    }
    // the columns past 3R
    for (int i = (warp - 4) * 32 + lane; i < (kN - 3 * R) * D / 4; i += 128)
      asm volatile("st.shared.u32 [%0], %1;" ::"r"(sQ + swizzled<D>(3 * R + 4 * i / D, 4 * i % D)), "r"(0u) : "memory");
    for (int i = (warp - 4) * 32 + lane; i < 2 * (kN - 3 * R) * kTile / 4; i += 128) {
      const int buf = i / ((kN - 3 * R) * kTile / 4 + (kN == 3 * R)), j = i - buf * ((kN - 3 * R) * kTile / 4);
      asm volatile("st.shared.u32 [%0], %1;" ::"r"(sP + buf * kN * kTile +
                                                   swizzled<128>(3 * R + 4 * j / kTile, 4 * j % kTile)),
                   "r"(0u)
                   : "memory");
    }
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;  // S at columns 0, kN; O^T at 2 kN, 3 kN

  if (warp < 4) {
    // ================================================================ softmax
    float vref = 0.f;
    for (int i = lane; i < n_blk; i += 32) vref = fmaxf(vref, s_vs[i]);
    vref = warp_max(vref);
    const float vmul = vref > 0.f ? kWeightScale / vref : 0.f;
    float m[R], l[R], qm[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      m[r] = -INFINITY;
      l[r] = 0.f;
      qm[r] = r < nr ? s_qm[r] : 0.f;
    }
    bool failed = false;
    for (int t = 0; t < n_t; ++t) {
      const int buf = t & 1, s = t % C::kStages;
      const int key = t * kTile + tid;
      const bool live = key < kn;
      const float ks = live ? s_ks[key >> 6] : 0.f, wv = live ? s_vs[key >> 6] * vmul : 0.f;
      if (!wait_all(bar_s + buf, (t >> 1) & 1, abort_flag, 3)) failed = true;
      tc_fence_after();
      uint32_t u[kN];
      tmem_ld_row<kN>(tmem + (static_cast<uint32_t>(warp * 32) << 16) + buf * kN, u);
      tc_fence_before();
      const bool edge = (t + 1) * kTile > lim_min;  // uniform: some row does not see the whole tile
      float x[R];
      bool big = false;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float sum = __uint_as_float(u[r]) + __uint_as_float(u[R + r]) + __uint_as_float(u[2 * R + r]);
        x[r] = sum * (qm[r] * ks);
        if (edge && key >= lim(r)) x[r] = -INFINITY;
        if (r >= nr) x[r] = -INFINITY;
        big = big || x[r] > m[r] + kMoveLog2;  // -inf > -inf: no
      }
      float al[R];
#pragma unroll
      for (int r = 0; r < R; ++r) al[r] = 1.f;
      if (softmax_bar_or(big || failed || *abort_flag)) {
        // some row's reference moves (or a wait gave up)
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float mx = warp_max(x[r]);  // NaN scores are left out: they show in p
          if (lane == 0) s_red[warp * R + r] = mx;
        }
        if (lane == 0) s_fail[warp] = failed || *abort_flag;
        softmax_bar();
        if (s_fail[0] | s_fail[1] | s_fail[2] | s_fail[3]) {
          *abort_flag = 1;
          break;
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float mx = fmaxf(fmaxf(s_red[r], s_red[R + r]), fmaxf(s_red[2 * R + r], s_red[3 * R + r]));
          if (mx > m[r] + kMoveLog2) {
            al[r] = m[r] == -INFINITY ? 0.f : ex2_approx(m[r] - mx);
            l[r] *= al[r];
            m[r] = mx;
          }
        }
      }
      // rows of V past the sequence may hold anything: they are cleared, so
      // that a weight of 0 adds exactly nothing.  A row that only some of the
      // new tokens see is cleared too if it holds a NaN, which its weight
      // then carries to the rows that do see it.
      float spoil = 0.f;
      if (edge) {
        if (!wait_all(bar_full + s, (t / C::kStages) & 1, abort_flag, 10)) failed = true;  // long done: S needed it
        const uint32_t vrow = smem_u32(smem + s * C::kStage + C::kOffV);
        bool clear = !live;
        if (live && key >= lim_min) {
          uint32_t nan = 0u;
#pragma unroll
          for (int c = 0; c < D; c += 16) {
            const uint4 w = ld_shared_v4(vrow + swizzled<D>(tid, c));
            nan |= ((w.x & 0x7f7f7f7fu) + 0x01010101u) | ((w.y & 0x7f7f7f7fu) + 0x01010101u) |
                   ((w.z & 0x7f7f7f7fu) + 0x01010101u) | ((w.w & 0x7f7f7f7fu) + 0x01010101u);
          }
          if (nan & 0x80808080u) {
            clear = true;
            spoil = NAN;
          }
        }
        if (clear) {
#pragma unroll
          for (int c = 0; c < D; c += 16) st_shared_v4(vrow + swizzled<D>(tid, c), 0u, 0u, 0u, 0u);
        }
      }
      // P and alpha of this buffer are free once tile t-2 is added up
      if (t >= 2 && !wait_all(bar_of + buf, ((t - 2) >> 1) & 1, abort_flag, 4)) failed = true;
      float w[R];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float pr = ex2_approx(x[r] - (m[r] == -INFINITY ? 0.f : m[r]));
        if (edge && key >= lim(r)) pr = 0.f;
        if (r >= nr) pr = 0.f;
        l[r] += pr;
        w[r] = pr * wv;
        if (edge && key < lim(r)) w[r] += spoil;
      }
      const uint32_t pcol = sP + buf * kN * kTile;
#pragma unroll
      for (int r = 0; r < R; r += 2) {
        float a = w[r], c = w[r + 1];
#pragma unroll
        for (int k = 0; k < 3; ++k) {
          const float ta = k < 2 ? lead3(a) : a, tc = k < 2 ? lead3(c) : c;
          const uint32_t two = e5m2x2(ta, tc);
          st_shared_u8(pcol + swizzled<128>(k * R + r, tid), two);
          st_shared_u8(pcol + swizzled<128>(k * R + r + 1, tid), two >> 8);
          a -= ta;
          c -= tc;
        }
      }
      if (tid < R) {
        float v = 1.f;
#pragma unroll
        for (int r = 0; r < R; ++r)
          if (tid == r) v = al[r];
        s_alpha[buf * R + tid] = v;
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_p + buf);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      l[r] = warp_sum(l[r]);
      if (lane == 0) s_l[warp * R + r] = l[r];
      if (tid == 0) s_m[r] = m[r];
    }
  } else if (warp < 8) {
    // ================================================================ output
    const int dd = tid - 128;
    if (dd < D) {
      float acc[R];
#pragma unroll
      for (int r = 0; r < R; ++r) acc[r] = 0.f;
      for (int t = 0; t < n_t; ++t) {
        const int buf = t & 1;
        // bar_p for alpha (the softmax warps' own arrivals), bar_o for O^T
        if (!wait_all(bar_p + buf, (t >> 1) & 1, abort_flag, 5)) break;
        if (!wait_all(bar_o + buf, (t >> 1) & 1, abort_flag, 5)) break;
        tc_fence_after();
        uint32_t u[kN];
        tmem_ld_row<kN>(tmem + (static_cast<uint32_t>((warp - 4) * 32) << 16) + (2 + buf) * kN, u);
        float al[R];
#pragma unroll
        for (int r = 0; r < R; ++r) al[r] = s_alpha[buf * R + r];
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_of + buf);
#pragma unroll
        for (int r = 0; r < R; ++r)
          acc[r] = fmaf(acc[r], al[r],
                        __uint_as_float(u[r]) + __uint_as_float(u[R + r]) + __uint_as_float(u[2 * R + r]));
      }
      // kept for after the barrier, over the stages (no longer read by then)
      asm volatile("bar.sync 2, 320;" ::: "memory");
      if (!*abort_flag) {
        float vref = 0.f;
        for (int i = 0; i < n_blk; ++i) vref = fmaxf(vref, s_vs[i]);
        const float osc = vref * (1.f / kWeightScale);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          if (r >= nr) break;
          const int tok = (row0 + r) / G, hq = hkv * G + (row0 + r) % G;
          const long long qrow = (static_cast<long long>(b) * p.Nq + tok) * p.Hq + hq;
          const float lr = (s_l[r] + s_l[R + r]) + (s_l[2 * R + r] + s_l[3 * R + r]);
          // l is 0 exactly where the row sees no key of the split (NaN, not 0, where a score is NaN)
          const float o = lr == 0.f ? 0.f : acc[r] * osc / lr;
          const float lse = lr == 0.f ? -INFINITY : (s_m[r] + __log2f(lr)) * 0.6931471805599453f;
          if (p.n_split == 1) {
            static_cast<__nv_bfloat16*>(p.o)[qrow * D + dd] = __float2bfloat16_rn(o);
            if (dd == 0) p.lse[(static_cast<long long>(b) * p.Hq + hq) * p.Nq + tok] = lse;
          } else {
            p.o_part[(qrow * p.n_split + split) * D + dd] = o;
            if (dd == 0) p.lse_part[qrow * p.n_split + split] = lse;
          }
        }
      }
    } else {
      asm volatile("bar.sync 2, 320;" ::: "memory");
    }
  } else if (warp == 8) {
    // ================================================================ loads
    if (lane == 0) {
      for (int t = C::kStages; t < n_t; ++t) {
        const int s = t % C::kStages;
        if (!wait_one(bar_empty + s, (t / C::kStages - 1) & 1, abort_flag, 6)) break;
        issue(t);
        n_issued = t + 1;
      }
    }
    __syncwarp();
  } else {
    // ================================================================ MMA
    if (lane == 0) {
      constexpr uint32_t idesc_s = idesc_e4m3_e5m2_f32(128, kN, 0), idesc_o = idesc_e4m3_e5m2_f32(128, kN, 1);
      auto desc = [](uint32_t addr, uint32_t lbo) {
        return D == 128 ? sdesc_sw128(addr, lbo, 1024) : sdesc_sw64(addr, lbo, 512);
      };
      auto scores = [&](int t) {
        const uint32_t k = smem_u32(smem + (t % C::kStages) * C::kStage + C::kOffK);
#pragma unroll
        for (int c = 0; c < D; c += 32)
          mma_f8_ss(tmem + (t & 1) * kN, desc(k + c, 16), desc(sQ + c, 16), idesc_s, c > 0);
        mma_commit(bar_s + (t & 1));
      };
      bool ok = n_t == 0 || wait_one(bar_full, 0, abort_flag, 7);
      tc_fence_after();
      if (ok && n_t > 0) scores(0);
      for (int t = 0; ok && t < n_t; ++t) {
        const int s = t % C::kStages;
        if (t + 1 < n_t) {
          ok = wait_one(bar_full + (t + 1) % C::kStages, ((t + 1) / C::kStages) & 1, abort_flag, 8);
          if (!ok) break;
          scores(t + 1);
        }
        ok = wait_one(bar_p + (t & 1), (t >> 1) & 1, abort_flag, 9);
        if (!ok) break;
        tc_fence_after();
        // V^T: M runs along the rows of the tile.  d = 64: M = 128 takes two
        // 64-dim blocks, of which the second (the K tile behind V, whatever
        // it holds) only reaches TMEM lanes that nothing reads.
        const uint32_t v = smem_u32(smem + s * C::kStage + C::kOffV), pb = sP + (t & 1) * kN * kTile;
#pragma unroll
        for (int c = 0; c < kTile; c += 32)
          mma_f8_ss(tmem + (2 + (t & 1)) * kN, desc(v + c * D, C::kTileBytes), sdesc_sw128(pb + c, 16, 1024), idesc_o,
                    c > 0);
        mma_commit(bar_o + (t & 1));
        mma_commit(bar_empty + s);
      }
      if (!ok) {
        // let the tensor core finish what was issued before TMEM goes (bounded, not abortable)
        volatile int no_abort = 0;
        mma_commit(bar_drain);
        mbar_wait(bar_drain, 0, &no_abort, kWaitLimitNs);
      }
    }
    __syncwarp();
  }
  if (warp == 8 && lane == 0 && *abort_flag) {
    // every issued load must land before the CTA may exit (bounded, not abortable)
    volatile int no_abort = 0;
    for (int t = n_issued > C::kStages ? n_issued - C::kStages : 0; t < n_issued; ++t)
      if (!mbar_wait(bar_full + (t % C::kStages), (t / C::kStages) & 1, &no_abort, kWaitLimitNs)) break;
  }
  if (warp < 4 || warp >= 8) asm volatile("bar.sync 2, 320;" ::: "memory");
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmem);
  }
}

// One block per row of q: LSE = ln sum_s exp(LSE_s), O = sum_s exp(LSE_s - LSE) O_s.
template <int D>
__global__ void __launch_bounds__(D) decode_fp8_combine_kernel(const DecodeFp8Params p) {
  const long long qrow = blockIdx.x;
  const int hq = static_cast<int>(qrow % p.Hq);
  const int i = static_cast<int>(qrow / p.Hq % p.Nq);
  const int b = static_cast<int>(qrow / p.Hq / p.Nq);
  const int dd = threadIdx.x;
  // launched as a programmatic dependent of the split kernel: wait until all
  // of its partials are written and visible
  asm volatile("griddepcontrol.wait;" ::: "memory");
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

template <int D, int R>
cudaError_t launch_rows(const DecodeFp8Params& p, cudaStream_t stream) {
  using C = Cfg<D, R>;
  auto kern = decode_fp8_split_kernel<D, R>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kAlloc);
  if (e != cudaSuccess) return e;
  const int rows = p.Nq * (p.Hq / p.Hkv);
  kern<<<dim3(p.Hkv * ((rows + R - 1) / R), p.B, p.n_split), kThreads, C::kAlloc, stream>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess || p.n_split == 1) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.B) * p.Nq * p.Hq);
  cfg.blockDim = dim3(D);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, decode_fp8_combine_kernel<D>, p);
}

template <int D>
cudaError_t launch_d(const DecodeFp8Params& p, cudaStream_t stream) {
  const int rows = p.Nq * (p.Hq / p.Hkv);
  if (rows <= 4) return launch_rows<D, 4>(p, stream);
  if (rows <= 8) return launch_rows<D, 8>(p, stream);
  return launch_rows<D, 16>(p, stream);
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

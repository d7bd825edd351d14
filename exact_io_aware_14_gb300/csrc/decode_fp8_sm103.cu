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
// Work items are (split of the keys, sequence, up to R query rows: heads of
// one KV head's group times new tokens).  A fixed grid of CTAs takes them in
// turn, full splits first, and keeps its pipeline running from one item to
// the next: with a CTA for each item, its start (lengths, pages, first loads)
// and end cost about 8 us each time, the time of 24 tiles of one SM.
// Eleven warps a CTA:
//   warps 0-3  softmax, a thread a key (TMEM lane): scales, running
//              reference, weights, their three terms as bytes into shared
//              memory
//   warps 4-7  output, a thread a dim: adds each tile's O^T columns to its
//              fp32 registers (so no rescaling in TMEM)
//   warp 8     items: finds them from the lengths, fetches their pages and
//              scales, turns q into e5m2 terms, up to kItems ahead
//   warp 9     TMEM, MMA issue: S of the next tile goes out before O of this
//              one where its K is there
//   warp 10    TMA loads, 128 keys of K and V a stage, in boxes of 64 rows
//              (pages are multiples of 64 rows)
// Two tiles of S, P and O are in flight.
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
constexpr int kThreads = 352;
constexpr uint64_t kWaitLimitNs = 2000000000ull;
constexpr float kMoveLog2 = 4.f;      // the reference moves when a score passes it by this
constexpr float kWeightScale = 1024.f;  // 2^10: weights up to 2^14, e5m2 ends at 57344

template <int D, int R>
struct Cfg {
  static constexpr int kN = (3 * R + 15) / 16 * 16;  // MMA columns
  static constexpr int kTmem = kN <= 16 ? 64 : (kN <= 32 ? 128 : 256);  // 4 kN, a power of two
  static constexpr int kCtas = R == 4 || (R == 8 && D == 64) ? 2 : 1;   // per SM
  static constexpr int kTileBytes = kTile * D;
  static constexpr int kStages = (kCtas == 2 ? 3 : (R == 16 ? 5 : 6)) * 128 / D - (D == 64 && R == 8 ? 1 : 0);
  static constexpr int kItems = 3;  // items prepared or in work
  static constexpr int kMaxBlocks = kMaxChunkFp8 / 64;
  static constexpr int kOffV = 0;  // V first: the M-major reads of a 64-dim V tile run into K's (see below)
  static constexpr int kOffK = kTileBytes;
  static constexpr int kStage = 2 * kTileBytes;
  static constexpr int kQBytes = (kN * D + 1023) / 1024 * 1024;
  static constexpr int kOffQ = kStages * kStage;            // [kItems]
  static constexpr int kOffP = kOffQ + kItems * kQBytes;    // [2][kN][128] bytes
  static constexpr int kOffItem = kOffP + 2 * kN * kTile;   // [kItems]
  static constexpr int kOffAlpha = kOffItem + kItems * ((12 + 3 * kMaxBlocks + R) * 4);  // float [2][R]
  static constexpr int kOffRed = kOffAlpha + 2 * R * 4;     // float [4][R], then 4 flags
  static constexpr int kOffMl = kOffRed + 4 * R * 4 + 16;   // [2] float m[R], l[4][R]
  static constexpr int kOffBar = (kOffMl + 2 * 5 * R * 4 + 15) / 16 * 16;
  static constexpr int kNumBars = 2 * kStages + 3 * kItems + 4 * 2 + 2 * 2 + 1;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kBytes = kOffMisc + 16;
  static constexpr int kAlloc = kBytes + 1024;
};

// One work item as the item warp hands it to the others.
template <int R>
struct Item {
  int n_t;       // key tiles; -1: no more items
  int kn;        // keys of the split
  int b, split, hkv, row0;
  int lim0;      // keys of the split that token 0 sees (may be negative or past kn)
  int direct;    // the sequence's only split: the result goes straight to o and lse
  float vref;    // largest value scale of the split
  int pad[3];
  int page[kMaxChunkFp8 / 64];  // of the split's 64-key blocks
  float ks[kMaxChunkFp8 / 64], vs[kMaxChunkFp8 / 64];
  float qm[R];   // softmax scale (base 2) over the row's power of two
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
__global__ void __launch_bounds__(kThreads, Cfg<D, R>::kCtas)
    decode_fp8_split_kernel(const __grid_constant__ DecodeFp8Params p) {
  using C = Cfg<D, R>;
  constexpr int kN = C::kN;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = p.Hq / p.Hkv;
  const int rows = p.Nq * G;  // query rows of a KV head: row r is token r / G, head r % G of the group

  Item<R>* items = reinterpret_cast<Item<R>*>(smem + C::kOffItem);
  static_assert(sizeof(Item<R>) == (12 + 3 * C::kMaxBlocks + R) * 4, "item size");
  float* s_alpha = reinterpret_cast<float*>(smem + C::kOffAlpha);
  float* s_red = reinterpret_cast<float*>(smem + C::kOffRed);
  int* s_fail = reinterpret_cast<int*>(smem + C::kOffRed + 4 * R * 4);
  float* s_ml = reinterpret_cast<float*>(smem + C::kOffMl);
  uint64_t* bar_full = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t* bar_empty = bar_full + C::kStages;
  uint64_t* bar_pages = bar_empty + C::kStages;  // [kItems] an item's description and pages are there
  uint64_t* bar_ready = bar_pages + C::kItems;   // [kItems] its scales and q too
  uint64_t* bar_free = bar_ready + C::kItems;    // [kItems] its readers are done (softmax, output, MMA, loads)
  uint64_t* bar_s = bar_free + C::kItems;        // [2] S of a tile in TMEM
  uint64_t* bar_p = bar_s + 2;                   // [2] P of a tile in shared memory (4 softmax warps)
  uint64_t* bar_o = bar_p + 2;                   // [2] O^T of a tile in TMEM
  uint64_t* bar_of = bar_o + 2;                  // [2] O^T and alpha read (D / 32 output warps)
  uint64_t* bar_ml = bar_of + 2;                 // [2] an item's m and l are there (4 softmax warps)
  uint64_t* bar_mf = bar_ml + 2;                 // [2] they were read (D / 32 output warps)
  uint64_t* bar_drain = bar_mf + 2;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
  const uint32_t sQ = smem_u32(smem + C::kOffQ), sP = smem_u32(smem + C::kOffP);

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (warp == 8) {
    if (lane == 0) {
      for (int s = 0; s < C::kStages; ++s) {
        mbar_init(bar_full + s, 1);
        mbar_init(bar_empty + s, 1);
      }
      for (int i = 0; i < C::kItems; ++i) {
        mbar_init(bar_pages + i, 1);
        mbar_init(bar_ready + i, 1);
        mbar_init(bar_free + i, 4 + D / 32 + 2);
      }
      for (int i = 0; i < 2; ++i) {
        mbar_init(bar_s + i, 1);
        mbar_init(bar_p + i, 4);
        mbar_init(bar_o + i, 1);
        mbar_init(bar_of + i, D / 32);
        mbar_init(bar_ml + i, 4);
        mbar_init(bar_mf + i, D / 32);
      }
      mbar_init(bar_drain, 1);
      *abort_flag = 0;
      mbar_fence_init();
    }
  } else if (warp == 9) {
    tmem_alloc(s_tmem, C::kTmem);
    tmem_relinquish();
  } else if (warp >= 4 && warp < 8) {
    // the MMA columns past 3R stay 0 in every Q and P
    constexpr int kPad = kN - 3 * R;
    for (int i = tid - 128; i < C::kItems * kPad * (D / 4); i += 128) {
      const int n = 3 * R + i / (D / 4) % (kPad + (kPad == 0)), slot = i / (D / 4) / (kPad + (kPad == 0));
      asm volatile("st.shared.u32 [%0], %1;" ::"r"(sQ + slot * C::kQBytes + swizzled<D>(n, 4 * (i % (D / 4)))), "r"(0u)
                   : "memory");
    }
    for (int i = tid - 128; i < 2 * kPad * (kTile / 4); i += 128) {
      const int n = 3 * R + i / (kTile / 4) % (kPad + (kPad == 0)), buf = i / (kTile / 4) / (kPad + (kPad == 0));
      asm volatile("st.shared.u32 [%0], %1;" ::"r"(sP + buf * kN * kTile + swizzled<128>(n, 4 * (i % (kTile / 4)))),
                   "r"(0u)
                   : "memory");
    }
    fence_proxy_async_smem();
  } else if (warp == 10 && lane == 0) {
    tma_prefetch_desc(&p.tm_k);
    tma_prefetch_desc(&p.tm_v);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;  // S at columns 0, kN; O^T at 2 kN, 3 kN
  int n_issued = 0;               // the loader's tiles

  if (warp < 4) {
    // ================================================================ softmax
    bool failed = false, stop = false;
    int g = 0;  // tiles so far, over all items
    for (int n = 0; !stop; ++n) {
      const Item<R>& it = items[n % C::kItems];
      if (!wait_all(bar_ready + n % C::kItems, (n / C::kItems) & 1, abort_flag, 3)) failed = true;
      if (softmax_bar_or(failed || *abort_flag)) {
        *abort_flag = 1;
        break;
      }
      const int n_t = it.n_t, kn = it.kn;
      if (n_t < 0) break;
      const int nr = min(R, rows - it.row0);
      // keys of the split that row r sees: those below lim(r)
      auto lim = [&](int r) { return min(kn, it.lim0 + (it.row0 + r) / G); };
      const int lim_min = lim(0);
      const float vmul = it.vref > 0.f ? kWeightScale / it.vref : 0.f;
      float m[R], l[R], qm[R];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        m[r] = -INFINITY;
        l[r] = 0.f;
        qm[r] = r < nr ? it.qm[r] : 0.f;
      }
      for (int t = 0; t < n_t; ++t, ++g) {
        const int buf = g & 1, s = g % C::kStages;
        const int key = t * kTile + tid;
        const bool live = key < kn;
        const float ks = live ? it.ks[key >> 6] : 0.f, wv = live ? it.vs[key >> 6] * vmul : 0.f;
        if (!wait_all(bar_s + buf, (g >> 1) & 1, abort_flag, 4)) failed = true;
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
            stop = true;
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
          // long done: S needed it
          if (!wait_all(bar_full + s, (g / C::kStages) & 1, abort_flag, 5)) failed = true;
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
        // P and alpha of this buffer are free once tile g-2 is added up
        if (g >= 2 && !wait_all(bar_of + buf, ((g - 2) >> 1) & 1, abort_flag, 6)) failed = true;
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
      if (stop) break;
      // m and l of the item, once the output warps have read those of item n-2
      if (n >= 2 && !wait_all(bar_mf + (n & 1), ((n >> 1) - 1) & 1, abort_flag, 7)) failed = true;
      float* ml = s_ml + (n & 1) * 5 * R;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        l[r] = warp_sum(l[r]);
        if (lane == 0) ml[(1 + warp) * R + r] = l[r];
        if (tid == 0) ml[r] = m[r];
      }
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar_ml + (n & 1));
        mbar_arrive(bar_free + n % C::kItems);
      }
    }
  } else if (warp < 8) {
    // ================================================================ output
    const int dd = tid - 128;
    if (dd < D) {
      int g = 0;
      bool ok = true;
      for (int n = 0; ok; ++n) {
        const Item<R>& it = items[n % C::kItems];
        if (!wait_all(bar_ready + n % C::kItems, (n / C::kItems) & 1, abort_flag, 8)) break;
        const int n_t = it.n_t;
        if (n_t < 0) break;
        float acc[R];
#pragma unroll
        for (int r = 0; r < R; ++r) acc[r] = 0.f;
        for (int t = 0; t < n_t; ++t, ++g) {
          const int buf = g & 1;
          // bar_p for alpha (the softmax warps' own arrivals), bar_o for O^T
          ok = wait_all(bar_p + buf, (g >> 1) & 1, abort_flag, 9) && wait_all(bar_o + buf, (g >> 1) & 1, abort_flag, 10);
          if (!ok) break;
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
        if (!ok || !wait_all(bar_ml + (n & 1), (n >> 1) & 1, abort_flag, 11)) break;
        const float* ml = s_ml + (n & 1) * 5 * R;
        const int nr = min(R, rows - it.row0), b = it.b, split = it.split, hkv = it.hkv, row0 = it.row0;
        const bool direct = it.direct != 0;
        const float osc = it.vref * (1.f / kWeightScale);
        float o[R], lse[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float lr = (ml[R + r] + ml[2 * R + r]) + (ml[3 * R + r] + ml[4 * R + r]);
          // l is 0 exactly where the row sees no key of the split (NaN, not 0, where a score is NaN)
          o[r] = lr == 0.f ? 0.f : acc[r] * osc / lr;
          lse[r] = lr == 0.f ? -INFINITY : (ml[r] + __log2f(lr)) * 0.6931471805599453f;
        }
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar_mf + (n & 1));
          mbar_arrive(bar_free + n % C::kItems);
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
          if (r >= nr) break;
          const int tok = (row0 + r) / G, hq = hkv * G + (row0 + r) % G;
          const long long qrow = (static_cast<long long>(b) * p.Nq + tok) * p.Hq + hq;
          if (direct) {
            static_cast<__nv_bfloat16*>(p.o)[qrow * D + dd] = __float2bfloat16_rn(o[r]);
            if (dd == 0) p.lse[(static_cast<long long>(b) * p.Hq + hq) * p.Nq + tok] = lse[r];
          } else {
            p.o_part[(qrow * p.n_split + split) * D + dd] = o[r];
            if (dd == 0) p.lse_part[qrow * p.n_split + split] = lse[r];
          }
        }
      }
    }
  } else if (warp == 8) {
    // ================================================================ items
    // Item i of the whole call: j = i / H counts (sequence, split) pairs, the
    // full splits of all sequences first and the shorter last ones after them,
    // i % H is the KV head and block of its rows (so neighbouring CTAs read
    // the same cache rows).  The lanes hold 32 sequences at a time; j only
    // grows, so they walk the batch once for the full splits and once for the
    // rest.
    const int n_rblk = (rows + R - 1) / R, H = p.Hkv * n_rblk;
    bool full_phase = true;
    int b0 = -32;
    long long before = 0;  // pairs before the lanes' sequences
    int Lb = 0, cnt = 0, excl = 0, total = 0;
    // next 32 sequences; false past the last
    auto next_block = [&]() {
      before += total;
      b0 += 32;
      if (b0 >= p.B) return false;
      Lb = b0 + lane < p.B ? p.seqlens[b0 + lane] : 0;
      if (Lb < 0 || Lb > p.max_seqlen) {
        record(1, kDevBadSeqlen);
        Lb = Lb < 0 ? 0 : p.max_seqlen;
      }
      if (full_phase)
        cnt = Lb / p.chunk;
      else  // with one split a sequence the empty ones are items too: nobody else writes their rows
        cnt = b0 + lane < p.B && (Lb % p.chunk > 0 || (Lb == 0 && p.n_split == 1)) ? 1 : 0;
      int incl = cnt;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      excl = incl - cnt;
      total = __shfl_sync(0xffffffffu, incl, 31);
      return true;
    };
    bool more = next_block();
    for (int n = 0;; ++n) {
      const int slot = n % C::kItems;
      Item<R>& it = items[slot];
      const long long i = blockIdx.x + static_cast<long long>(n) * gridDim.x, j = i / H;
      const int h = static_cast<int>(i - j * H);
      while (more && j >= before + total) {
        more = next_block();
        if (!more && full_phase) {
          full_phase = false;
          b0 = -32;
          total = 0;
          more = next_block();
        }
      }
      int b = 0, split = 0, len = 0;
      if (more) {
        const int rel = static_cast<int>(j - before);
        const unsigned who = __ballot_sync(0xffffffffu, cnt > 0 && rel >= excl && rel < excl + cnt);
        const int src = __ffs(who) - 1;
        b = b0 + src;
        len = __shfl_sync(0xffffffffu, Lb, src);
        split = full_phase ? rel - __shfl_sync(0xffffffffu, excl, src) : len / p.chunk;
      }
      if (n >= C::kItems && !wait_all(bar_free + slot, (n / C::kItems - 1) & 1, abort_flag, 12)) break;
      const int k0 = split * p.chunk, kn = min(p.chunk, len - k0), n_blk = (kn + 63) / 64;
      const int hkv = h / n_rblk, row0 = (h - hkv * n_rblk) * R;
      if (lane == 0) {
        it.n_t = more ? (kn + kTile - 1) / kTile : -1;
        it.kn = kn;
        it.b = b;
        it.split = split;
        it.hkv = hkv;
        it.row0 = row0;
        it.lim0 = len - p.Nq + 1 - k0;
        it.direct = len <= p.chunk;
      }
      int pg[C::kMaxBlocks / 32];
      if (more) {
#pragma unroll
        for (int k = 0; k < C::kMaxBlocks / 32; ++k) {
          const int blk = 32 * k + lane;
          pg[k] = 0;
          if (blk < n_blk) {
            pg[k] = p.block_table[static_cast<long long>(b) * p.max_blocks + (k0 + 64 * blk) / p.page_size];
            if (pg[k] < 0 || pg[k] >= p.num_pages) {
              record(2, kDevBadPage);
              pg[k] = 0;  // keep every load inside the page pool; the result is flagged
            }
            it.page[blk] = pg[k];
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_pages + slot);
      if (more) {
        float vref = 0.f;
#pragma unroll
        for (int k = 0; k < C::kMaxBlocks / 32; ++k) {
          const int blk = 32 * k + lane;
          if (blk < n_blk) {
            it.ks[blk] = p.k_scales[static_cast<long long>(pg[k]) * p.Hkv + hkv];
            const float vs = p.v_scales[static_cast<long long>(pg[k]) * p.Hkv + hkv];
            it.vs[blk] = vs;
            vref = fmaxf(vref, vs);
          }
        }
        vref = warp_max(vref);
        if (lane == 0) it.vref = vref;
        // q as three e5m2 terms a row: column term * R + r
        const int nr = min(R, rows - row0);
        const uint32_t q_at = sQ + slot * C::kQBytes;
        float x[R][D / 32];
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const int tok = (row0 + r) / G, hq = hkv * G + (row0 + r) % G;
#pragma unroll
          for (int i2 = 0; i2 < D / 32; i2 += 2) {
            uint32_t two = 0u;
            if (r < nr)
              two = *reinterpret_cast<const uint32_t*>(
                  static_cast<const __nv_bfloat16*>(p.q) +
                  ((static_cast<long long>(b) * p.Nq + tok) * p.Hq + hq) * D + (D / 32) * lane + i2);
            x[r][i2] = bf16lo(two);
            x[r][i2 + 1] = bf16hi(two);
          }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
          float amax = 0.f;
          bool fin = true;
#pragma unroll
          for (int i2 = 0; i2 < D / 32; ++i2) {
            fin = fin && fabsf(x[r][i2]) < INFINITY;
            amax = fmaxf(amax, fabsf(x[r][i2]));
          }
          amax = warp_max(amax);
          fin = __all_sync(0xffffffffu, fin);
          const int e = fin ? max(static_cast<int>(__float_as_uint(amax) >> 23) - 127, -100) : 0;
          const float f = __uint_as_float(static_cast<uint32_t>(14 - e + 127) << 23);
          uint32_t term[3] = {0u, 0u, 0u};
#pragma unroll
          for (int i2 = 0; i2 < D / 32; i2 += 2) {
            float a = fin ? x[r][i2] * f : 0.f, c = fin ? x[r][i2 + 1] * f : 0.f;
#pragma unroll
            for (int k = 0; k < 3; ++k) {
              const float ta = lead3(a), tc = lead3(c);
              term[k] |= e5m2x2(ta, tc) << (8 * i2);
              a -= ta;
              c -= tc;
            }
          }
#pragma unroll
          for (int k = 0; k < 3; ++k) {
            const uint32_t at = q_at + swizzled<D>(k * R + r, (D / 32) * lane);
            if (D == 128)
              asm volatile("st.shared.u32 [%0], %1;" ::"r"(at), "r"(term[k]) : "memory");
            else
              asm volatile("st.shared.u16 [%0], %1;" ::"r"(at), "h"(static_cast<uint16_t>(term[k])) : "memory");
          }
          // a row with an infinity or NaN: every score NaN
          if (lane == 0)
            it.qm[r] = fin ? __uint_as_float(static_cast<uint32_t>(e - 14 + 127) << 23) * p.scale_log2 : NAN;
        }
        fence_proxy_async_smem();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_ready + slot);
      if (!more) break;
    }
  } else if (warp == 9) {
    // ================================================================ MMA
    if (lane == 0) {
      constexpr uint32_t idesc_s = idesc_e4m3_e5m2_f32(128, kN, 0), idesc_o = idesc_e4m3_e5m2_f32(128, kN, 1);
      auto desc = [](uint32_t addr, uint32_t lbo) {
        return D == 128 ? sdesc_sw128(addr, lbo, 1024) : sdesc_sw64(addr, lbo, 512);
      };
      // tile gn of the CTA, of item n: S = K Q^T
      auto scores = [&](int gn, int n) {
        const uint32_t k = smem_u32(smem + (gn % C::kStages) * C::kStage + C::kOffK);
        const uint32_t q = sQ + (n % C::kItems) * C::kQBytes;
#pragma unroll
        for (int c = 0; c < D; c += 32)
          mma_f8_ss(tmem + (gn & 1) * kN, desc(k + c, 16), desc(q + c, 16), idesc_s, c > 0);
        mma_commit(bar_s + (gn & 1));
      };
      bool ok = true;
      int n = -1, left = 0;  // current item of the S side, its tiles still to issue
      // moves to the next tile; `block`: waits for its item, else gives up if
      // that is not there yet.  1: there is one, 0: no more, -1: not there
      auto next_tile = [&](bool block) {
        while (left == 0) {
          uint64_t* bar = bar_ready + (n + 1) % C::kItems;
          const uint32_t par = ((n + 1) / C::kItems) & 1;
          if (block) {
            if (!wait_one(bar, par, abort_flag, 13)) {
              ok = false;
              return 0;
            }
          } else if (!mbar_test_wait(bar, par)) {
            return -1;
          }
          const int n_t = items[(n + 1) % C::kItems].n_t;
          if (n_t < 0) return 0;
          ++n;
          left = n_t;
          mbar_arrive(bar_free + n % C::kItems);  // only the count was read; Q is given back by the softmax warps
        }
        return 1;
      };
      int g = 0;
      int have = next_tile(true);
      if (ok && have == 1) {
        ok = wait_one(bar_full, 0, abort_flag, 14);
        tc_fence_after();
        if (ok) {
          scores(0, n);
          --left;
        }
      }
      while (ok && have == 1) {  // S of tile g is issued
        const int s = g % C::kStages, s1 = (g + 1) % C::kStages;
        const uint32_t par1 = ((g + 1) / C::kStages) & 1;
        have = next_tile(false);
        bool issued = false;
        if (have == 1 && mbar_test_wait(bar_full + s1, par1)) {
          scores(g + 1, n);
          --left;
          issued = true;
        }
        ok = wait_one(bar_p + (g & 1), (g >> 1) & 1, abort_flag, 15);
        if (!ok) break;
        tc_fence_after();
        // V^T: M runs along the rows of the tile.  d = 64: M = 128 takes two
        // 64-dim blocks, of which the second (the K tile behind V, whatever
        // it holds) only reaches TMEM lanes that nothing reads.
        const uint32_t v = smem_u32(smem + s * C::kStage + C::kOffV), pb = sP + (g & 1) * kN * kTile;
#pragma unroll
        for (int c = 0; c < kTile; c += 32)
          mma_f8_ss(tmem + (2 + (g & 1)) * kN, desc(v + c * D, C::kTileBytes), sdesc_sw128(pb + c, 16, 1024), idesc_o,
                    c > 0);
        mma_commit(bar_o + (g & 1));
        mma_commit(bar_empty + s);
        if (!issued) {
          if (have < 0) have = next_tile(true);
          if (ok && have == 1) {
            ok = wait_one(bar_full + s1, par1, abort_flag, 16);
            if (!ok) break;
            scores(g + 1, n);
            --left;
          }
        }
        ++g;
      }
      if (!ok) {
        // let the tensor core finish what was issued before TMEM goes (bounded, not abortable)
        volatile int no_abort = 0;
        mma_commit(bar_drain);
        mbar_wait(bar_drain, 0, &no_abort, kWaitLimitNs);
      }
    }
    __syncwarp();
  } else {
    // ================================================================ loads
    if (lane == 0) {
      bool ok = true;
      for (int n = 0; ok; ++n) {
        const Item<R>& it = items[n % C::kItems];
        if (!wait_one(bar_pages + n % C::kItems, (n / C::kItems) & 1, abort_flag, 17)) break;
        const int n_t = it.n_t, n_blk = (it.kn + 63) / 64, hkv = it.hkv, k0 = it.split * p.chunk;
        if (n_t < 0) break;
        for (int t = 0; t < n_t; ++t) {
          const int g = n_issued, s = g % C::kStages;
          if (g >= C::kStages && !wait_one(bar_empty + s, (g / C::kStages - 1) & 1, abort_flag, 18)) {
            ok = false;
            break;
          }
          const int nb = min(2, n_blk - 2 * t);
          mbar_arrive_expect_tx(bar_full + s, 2 * nb * 64 * D);
          for (int i = 0; i < nb; ++i) {
            const int blk = 2 * t + i, row = (k0 + 64 * blk) % p.page_size, page = it.page[blk];
            tma_load_4d(smem + s * C::kStage + C::kOffK + i * 64 * D, &p.tm_k, bar_full + s, 0, hkv, row, page);
            tma_load_4d(smem + s * C::kStage + C::kOffV + i * 64 * D, &p.tm_v, bar_full + s, 0, hkv, row, page);
          }
          n_issued = g + 1;
        }
        if (ok) mbar_arrive(bar_free + n % C::kItems);
      }
      if (*abort_flag) {
        // every issued load must land before the CTA may exit (bounded, not abortable)
        volatile int no_abort = 0;
        for (int t = n_issued > C::kStages ? n_issued - C::kStages : 0; t < n_issued; ++t)
          if (!mbar_wait(bar_full + (t % C::kStages), (t / C::kStages) & 1, &no_abort, kWaitLimitNs)) break;
      }
    }
    __syncwarp();
  }
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmem);
  }
}

// One block of 8 warps per row of q: LSE = ln sum_s exp(LSE_s), O = sum_s
// exp(LSE_s - LSE) O_s.  A warp takes every eighth split, D/32 values a lane,
// four splits' loads in flight; the warps' sums are added in a fixed order.
constexpr int kCombineWarps = 8;

template <int D>
__global__ void __launch_bounds__(32 * kCombineWarps) decode_fp8_combine_kernel(const DecodeFp8CombineParams p) {
  constexpr int kV = D / 32;
  __shared__ float s_max[kCombineWarps], s_tot[kCombineWarps];
  __shared__ float s_acc[kCombineWarps][D];
  const long long qrow = blockIdx.x;
  const int hq = static_cast<int>(qrow % p.Hq);
  const int i = static_cast<int>(qrow / p.Hq % p.Nq);
  const int b = static_cast<int>(qrow / p.Hq / p.Nq);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // launched as a programmatic dependent of the split kernel: wait until all
  // of its partials are written and visible
  asm volatile("griddepcontrol.wait;" ::: "memory");
  int Lb = p.seqlens[b];
  Lb = Lb < 0 ? 0 : (Lb > p.max_seqlen ? p.max_seqlen : Lb);
  const int ns = (Lb + p.chunk - 1) / p.chunk;
  if (ns == 1) return;  // written by the split kernel
  const float* lp = p.lse_part + qrow * p.n_split;
  const float* op = p.o_part + qrow * p.n_split * D + kV * lane;
  float mx = -INFINITY;
  for (int s = threadIdx.x; s < ns; s += 32 * kCombineWarps) mx = fmaxf(mx, lp[s]);
  mx = warp_max(mx);
  if (lane == 0) s_max[warp] = mx;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kCombineWarps; ++w) mx = fmaxf(mx, s_max[w]);
  if (mx == -INFINITY) mx = 0.f;  // no key seen (or every LSE NaN): the weights are then 0 (NaN)
  float tot = 0.f, acc[kV];
#pragma unroll
  for (int k = 0; k < kV; ++k) acc[k] = 0.f;
  for (int s = warp; s < ns; s += 4 * kCombineWarps) {
    float lv[4], ov[4][kV];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int su = s + u * kCombineWarps;
      lv[u] = su < ns ? lp[su] : -INFINITY;
#pragma unroll
      for (int k = 0; k < kV; ++k) ov[u][k] = 0.f;
      if (su < ns) {
        if (kV == 4) {
          const float4 v = *reinterpret_cast<const float4*>(op + static_cast<long long>(su) * D);
          ov[u][0] = v.x; ov[u][1] = v.y; ov[u][kV - 2] = v.z; ov[u][kV - 1] = v.w;
        } else {
          const float2 v = *reinterpret_cast<const float2*>(op + static_cast<long long>(su) * D);
          ov[u][0] = v.x; ov[u][1] = v.y;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const float w = expf(lv[u] - mx);
      tot += w;
#pragma unroll
      for (int k = 0; k < kV; ++k) acc[k] = fmaf(w, ov[u][k], acc[k]);
    }
  }
  if (lane == 0) s_tot[warp] = tot;
#pragma unroll
  for (int k = 0; k < kV; ++k) s_acc[warp][kV * lane + k] = acc[k];
  __syncthreads();
  if (threadIdx.x >= D) return;
  float a = 0.f, sum = 0.f;
#pragma unroll
  for (int w = 0; w < kCombineWarps; ++w) {
    a += s_acc[w][threadIdx.x];
    sum += s_tot[w];
  }
  const bool none = sum == 0.f;
  static_cast<__nv_bfloat16*>(p.o)[qrow * D + threadIdx.x] = __float2bfloat16_rn(none ? 0.f : a / sum);
  if (threadIdx.x == 0) p.lse[(static_cast<long long>(b) * p.Hq + hq) * p.Nq + i] = none ? -INFINITY : mx + logf(sum);
}

template <int D, int R>
cudaError_t launch_rows(const DecodeFp8Params& p, int sms, cudaStream_t stream) {
  using C = Cfg<D, R>;
  auto kern = decode_fp8_split_kernel<D, R>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kAlloc);
  if (e != cudaSuccess) return e;
  const int rows = p.Nq * (p.Hq / p.Hkv);
  const long long items = static_cast<long long>(p.Hkv) * ((rows + R - 1) / R) * p.B * p.n_split;
  const long long ctas = static_cast<long long>(sms) * C::kCtas;
  kern<<<static_cast<unsigned>(items < ctas ? items : ctas), kThreads, C::kAlloc, stream>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess || p.n_split == 1) return e;
  const DecodeFp8CombineParams c = {p.o_part, p.lse_part, p.seqlens, p.o, p.lse, p.Nq, p.Hq, p.max_seqlen, p.chunk,
                                    p.n_split};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.B) * p.Nq * p.Hq);
  cfg.blockDim = dim3(32 * kCombineWarps);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, decode_fp8_combine_kernel<D>, c);
}

template <int D>
cudaError_t launch_d(const DecodeFp8Params& p, cudaStream_t stream) {
  int dev, sms;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int rows = p.Nq * (p.Hq / p.Hkv);
  if (rows <= 4) return launch_rows<D, 4>(p, sms, stream);
  if (rows <= 8) return launch_rows<D, 8>(p, sms, stream);
  return launch_rows<D, 16>(p, sms, stream);
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

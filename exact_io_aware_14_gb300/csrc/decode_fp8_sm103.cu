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
// 3R columns, the three terms of a row are added up in fp32 afterwards.  Four
// terms a weight brought outputs from 0.0012 to 0.0004 of those with 32-bit
// weights, under the 0.0017 of their own rounding to bf16, and took 58.2 us for
// 57.2 on a serving batch, 107 for 100 where there are 24 rows (d = 128).
// q is scaled by a power of two a row (largest value in [2^14, 2^15)).  The
// weights p = 2^(s - m) enter the second product as p v 2^10, v the page's
// value scale over the split's largest.  The running reference m follows the
// largest s + ceil(log2 v), not the largest score, and moves when a key passes
// it by 4: so the largest p v 2^10 of a row is in (2^9, 2^14], however far the
// pages' scales lie apart, and what e5m2 drops below 2^-17 is under 2^-26 of
// it.  p itself, which only the sum of weights sees, may be as large as 2^104
// (log2 v counts down to -100).
//
// Work items are (split of the keys, sequence, up to R query rows: heads of
// one KV head's group times new tokens).  A fixed grid of CTAs takes them in
// turn, full splits first, and keeps its pipeline running from one item to
// the next: with a CTA for each item, its start (lengths, pages, first loads)
// and end cost about 8 us each time, the time of 24 tiles of one SM.  Which
// items a CTA takes is fixed (SMs end up to 15% apart; claiming items from a
// counter evened that out, but clearing the counter took a launch, and the
// two cancelled: 55.1 and 56.9 us on a serving batch, 182 and 181 us on two
// sequences of 256 K keys).
// The warps of a CTA, in this order:
//   softmax    one to three groups of four warps, a thread a key (TMEM lane):
//              scales, running reference, weights, their three terms as bytes
//              into shared memory
//   output     two or four warps, a thread a dim: adds each tile's O^T columns to its
//              fp32 registers (so no rescaling in TMEM)
//   items      one to three warps: find them from the lengths, fetch their pages
//              and scales, turn q into e5m2 terms, up to kItems ahead
//   MMA        one warp: TMEM, MMA issue; S of the next tile goes out before O
//              of this one where its K is there
//   loads      one warp: TMA, 128 keys of K and V a stage, in boxes of 64 rows
//              (pages are multiples of 64 rows)
// Two tiles of S, P and O are in flight.
//
// Where the splits of a group of rows are two to eight and there is a place on an
// SM for every CTA, they form a cluster instead, a CTA a split, and combine their
// results through distributed shared memory: no second kernel.  (Clusters do not
// wait for one another, so those that find no group of SMs free take their turn.)
//
// Combine kernel: LSE = ln sum_s exp(LSE_s), O = sum_s exp(LSE_s - LSE) O_s.
#include <atomic>

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
constexpr uint64_t kWaitLimitNs = 2000000000ull;
constexpr float kMoveLog2 = 4.f;      // the reference moves when a key passes it by this
constexpr int kNoKey = 0x7fffffff;
constexpr float kWeightScale = 1024.f;  // 2^10: weights up to 2^14, e5m2 ends at 57344

template <int D, int R>
struct Cfg {
  static constexpr int kN = (3 * R + 15) / 16 * 16;  // MMA columns
  static constexpr int kTmem = kN <= 16 ? 64 : (kN <= 32 ? 128 : (kN <= 64 ? 256 : 512));  // 4 kN, a power of two
  static constexpr int kCtas = R == 4 ? 2 : 1;                          // per SM
  // softmax groups of four warps, each with its own kRows of the rows: a group
  // takes about 0.5 us for a tile of four rows and 0.9 us for eight; at HBM rate
  // a tile of d = 128 arrives every 0.72 us on an SM
  static constexpr int kGroups = R == 4 ? 1 : (R == 24 ? 3 : 2);
  static constexpr int kRows = R / kGroups;
  static constexpr int kSoftWarps = 4 * kGroups;
  static constexpr int kOutWarps = D / 32;
  // warps that prepare items, each 8 rows of q (4 of R = 4): one warp took 5 us
  // for 24 rows, the time of five tiles.  20 warps at most, for 96 registers.
  static constexpr int kItemWarps = R <= 8 ? 1 : (R == 24 && D == 128 ? 2 : R / 8);
  static constexpr int kWarps = kSoftWarps + kOutWarps + kItemWarps + 2;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kTileBytes = kTile * D;
  static constexpr int kStages = (kCtas == 2 ? 3 : (R == 8 ? 6 : 5)) * 128 / D;
  static constexpr int kItems = R == 24 ? 3 : 4;  // items prepared or in work
  static constexpr int kMaxBlocks = kMaxChunkFp8 / 64;
  static constexpr int kOffV = 0;  // V first: the M-major reads of a 64-dim V tile run into K's (see below)
  static constexpr int kOffK = kTileBytes;
  static constexpr int kStage = 2 * kTileBytes;
  static constexpr int kQBytes = (kN * D + 1023) / 1024 * 1024;
  static constexpr int kOffQ = kStages * kStage;            // [kItems]
  static constexpr int kOffP = kOffQ + kItems * kQBytes;    // [2] kN x 128 bytes (p_at)
  static constexpr int kOffItem = kOffP + 2 * kN * kTile;   // [kItems]
  static constexpr int kOffAlpha = kOffItem + kItems * ((8 + 3 * kMaxBlocks + 4 * R) * 4);  // float [2][R]
  static constexpr int kOffRed = kOffAlpha + 2 * R * 4;     // [kGroups] float [4][kRows], then [kGroups] 4 flags
  static_assert(kRows == 4 || kRows == 8, "stored as words");
  static_assert(kOffRed % 16 == 0, "read four rows at a time");
  static constexpr int kOffNan = kOffRed + 4 * R * 4 + kGroups * 16;  // int [2][D]
  static constexpr int kOffMl = kOffNan + 2 * D * 4;        // [2] float m[R], l[4][R]
  static constexpr int kOffBar = (kOffMl + 2 * 5 * R * 4 + 15) / 16 * 16;
  static constexpr int kNumBars = 2 * kStages + 3 * kItems + 4 * 2 + 2 * 2 + 1;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kBytes = kOffMisc + 16;
  static constexpr int kAlloc = kBytes + 1024;
  static_assert(kCtas * (kAlloc + 1024) <= 228 * 1024, "an SM's shared memory, 1 KB of it reserved for each CTA");
};

// One work item as the item warp hands it to the others.
template <int R>
struct Item {
  int n_t;       // key tiles; -1: no more items
  int kn;        // keys of the split
  int split, hkv;
  int lim_min;   // keys of the split that every row sees, at least
  int direct;    // the sequence's only split: the result goes straight to o and lse
  float vref;    // largest value scale of the split
  int pad[1];
  int page[kMaxChunkFp8 / 64];  // of the split's 64-key blocks
  float ks[kMaxChunkFp8 / 64];
  float vs[kMaxChunkFp8 / 64];  // over vref, times kWeightScale
  float qm[R];   // softmax scale (base 2) over the row's power of two
  int lim[R];    // keys of the split that row r sees: those below lim[r] (0 or less: none)
  int o_row[R], lse_row[R];  // where its results go, in rows of o and entries of lse; -1: no such row
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

// named barrier over the four warps of a softmax group, with an OR of a flag
__device__ __forceinline__ bool softmax_bar_or(int group, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred pi, po;\n\t"
      "setp.ne.u32 pi, %1, 0;\n\t"
      "bar.red.or.pred po, %2, 128, pi;\n\t"
      "selp.u32 %0, 1, 0, po;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(v)), "r"(1 + group)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void softmax_bar(int group) {
  asm volatile("bar.sync %0, 128;" ::"r"(1 + group) : "memory");
}

// two floats -> two e5m2 codes, `lo` in the low byte
__device__ __forceinline__ uint32_t e5m2x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// x cut to its 3 leading significant bits (what one e5m2 term holds)
__device__ __forceinline__ float lead3(float x) { return __uint_as_float(__float_as_uint(x) & 0xffe00000u); }

// Largest values of kN rows (4 or 8) over the warp, NaN left out: each step
// halves the rows a lane holds, then the lanes of a row are reduced.  Returns
// row lane / (32 / kN)'s.
template <int kN>
__device__ __forceinline__ float warp_max_rows(float (&v)[kN]) {
  const int lane = threadIdx.x & 31;
  int o = 16;
#pragma unroll
  for (int half = kN / 2; half > 0; half /= 2, o /= 2) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < half; ++i) {
      const float give = up ? v[i] : v[half + i], keep = up ? v[half + i] : v[i];
      v[i] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, give, o));
    }
  }
#pragma unroll
  for (; o > 0; o /= 2) v[0] = fmaxf(v[0], __shfl_xor_sync(0xffffffffu, v[0], o));
  return v[0];
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

// MMA column of term k of row r: the rows of a softmax group lie together.
template <int R, int kRows>
__device__ __forceinline__ constexpr int column(int k, int r) {
  return r / kRows * 3 * kRows + k * kRows + r % kRows;
}

// ceil(log2 v) of wv = v * kWeightScale, v in [0, 1]; -100 at the least.
__device__ __forceinline__ float log2_up(float wv) {
  const uint32_t u = __float_as_uint(wv);
  return static_cast<float>(max(static_cast<int>(u >> 23) - (127 + 10) + ((u & 0x7fffffu) != 0u ? 1 : 0), -100));
}

// Byte offset of row n, byte c of an operand with rows of D bytes, swizzled
// as TMA and the MMA descriptors have it.
template <int kRow>
__device__ __forceinline__ int swizzled(int n, int c) {
  const int chunk = (c >> 4) ^ (kRow == 128 ? (n & 7) : ((n >> 1) & 3));
  return n * kRow + (chunk << 4) + (c & 15);
}

// Byte offset of column n of key k in P (N-major without swizzle: a key's
// columns lie together in 16-byte pieces, so a thread writes a term of all its
// rows at once; with K-major rows it wrote each byte by itself, 24 stores a
// tile for eight rows).
__device__ __forceinline__ int p_at(int n, int k) { return (n >> 4) * (16 * kTile) + k * 16 + (n & 15); }

// The first kN (at least) columns of this thread's TMEM lane from addr on.
template <int kN>
__device__ __forceinline__ void tmem_ld_row(uint32_t addr, uint32_t (&u)[kN]) {
#pragma unroll
  for (int c = 0; c + 16 <= kN; c += 16) tmem_ld16(addr + c, u + c);
  if (kN % 16 == 8) tmem_ld8(addr + kN / 16 * 16, u + kN / 16 * 16);
  tmem_wait_ld();
}

template <int D, int R>
__global__ void __launch_bounds__(Cfg<D, R>::kThreads, Cfg<D, R>::kCtas)
    decode_fp8_split_kernel(const __grid_constant__ DecodeFp8Params p) {
  using C = Cfg<D, R>;
  constexpr int kN = C::kN, kRows = C::kRows, kOut0 = C::kSoftWarps;  // kOut0: the first output warp
  constexpr int kItemWarp = kOut0 + C::kOutWarps, kMmaWarp = kItemWarp + C::kItemWarps, kLoadWarp = kMmaWarp + 1;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rows = p.rows;  // query rows of a KV head: row r is token r / G, head r % G of the group of G heads

  Item<R>* items = reinterpret_cast<Item<R>*>(smem + C::kOffItem);
  static_assert(sizeof(Item<R>) == (8 + 3 * C::kMaxBlocks + 4 * R) * 4, "item size");
  float* s_alpha = reinterpret_cast<float*>(smem + C::kOffAlpha);
  float* s_red = reinterpret_cast<float*>(smem + C::kOffRed);
  int* s_fail = reinterpret_cast<int*>(smem + C::kOffRed + 4 * R * 4);
  int* s_nan = reinterpret_cast<int*>(smem + C::kOffNan);  // first key of a tile whose value has a NaN in a dim
  float* s_ml = reinterpret_cast<float*>(smem + C::kOffMl);
  uint64_t* bar_full = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t* bar_empty = bar_full + C::kStages;
  uint64_t* bar_pages = bar_empty + C::kStages;  // [kItems] an item's description and pages are there
  uint64_t* bar_ready = bar_pages + C::kItems;   // [kItems] its scales and q too
  uint64_t* bar_free = bar_ready + C::kItems;    // [kItems] its readers are done (softmax, output, MMA, loads)
  uint64_t* bar_s = bar_free + C::kItems;        // [2] S of a tile in TMEM
  uint64_t* bar_p = bar_s + 2;                   // [2] P of a tile in shared memory (the softmax warps)
  uint64_t* bar_o = bar_p + 2;                   // [2] O^T of a tile in TMEM
  uint64_t* bar_of = bar_o + 2;                  // [2] O^T and alpha read (D / 32 output warps)
  uint64_t* bar_ml = bar_of + 2;                 // [2] an item's m and l are there (the softmax warps)
  uint64_t* bar_mf = bar_ml + 2;                 // [2] they were read (D / 32 output warps)
  uint64_t* bar_drain = bar_mf + 2;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
  const uint32_t sQ = smem_u32(smem + C::kOffQ), sP = smem_u32(smem + C::kOffP);

  grid_release();
  if (warp == kLoadWarp) {
    if (lane == 0) {
      tma_prefetch_desc(&p.tm_k);
      tma_prefetch_desc(&p.tm_v);
      for (int s = 0; s < C::kStages; ++s) {
        mbar_init(bar_full + s, 1);
        mbar_init(bar_empty + s, 1);
      }
      for (int i = 0; i < C::kItems; ++i) {
        mbar_init(bar_pages + i, 1);
        mbar_init(bar_ready + i, C::kItemWarps);
        mbar_init(bar_free + i, C::kSoftWarps + D / 32 + 2);
      }
      for (int i = 0; i < 2; ++i) {
        mbar_init(bar_s + i, 1);
        mbar_init(bar_p + i, C::kSoftWarps);
        mbar_init(bar_o + i, 1);
        mbar_init(bar_of + i, D / 32);
        mbar_init(bar_ml + i, C::kSoftWarps);
        mbar_init(bar_mf + i, D / 32);
      }
      mbar_init(bar_drain, 1);
      *abort_flag = 0;
      mbar_fence_init();
    }
  } else if (warp >= kOut0 && warp < kItemWarp) {
    // the MMA columns past 3R stay 0 in every Q and P
    constexpr int kPad = kN - 3 * R;
    for (int i = tid - 32 * kOut0; i < C::kItems * kPad * (D / 4); i += D) {
      const int n = 3 * R + i / (D / 4) % (kPad + (kPad == 0)), slot = i / (D / 4) / (kPad + (kPad == 0));
      asm volatile("st.shared.u32 [%0], %1;" ::"r"(sQ + slot * C::kQBytes + swizzled<D>(n, 4 * (i % (D / 4)))), "r"(0u)
                   : "memory");
    }
    for (int i = tid - 32 * kOut0; i < 2 * kPad / 4 * kTile; i += D) {
      const int n = 3 * R + i / kTile % (kPad / 4 + (kPad == 0)) * 4, buf = i / kTile / (kPad / 4 + (kPad == 0));
      asm volatile("st.shared.u32 [%0], %1;" ::"r"(sP + buf * kN * kTile + p_at(n, i % kTile)), "r"(0u) : "memory");
    }
    s_nan[tid - 32 * kOut0] = s_nan[D + tid - 32 * kOut0] = kNoKey;
    fence_proxy_async_smem();
  }
  // clustered: this split's result, in the place of the first stages
  float* s_part = reinterpret_cast<float*>(smem);
  float* s_part_lse = s_part + R * D;
  int* s_part_row = reinterpret_cast<int*>(s_part_lse + R);  // rows of o, then entries of lse
  static_assert((R * D + 3 * R) * 4 <= C::kStages * C::kStage, "a split's result fits the stages");

  // Launched as a programmatic dependent of whatever ran before: nothing of that
  // is read before this wait, and no Tensor Memory is held during it (the kernel
  // before may have CTAs that are still to ask for theirs), nor does the limit of
  // any wait below run.
  grid_wait();
  if (warp == kMmaWarp) {
    tmem_alloc(s_tmem, C::kTmem);
    tmem_relinquish();
  }
  uint32_t tmem = 0u;  // S at columns 0, kN; O^T at 2 kN, 3 kN
  if (warp < kItemWarp || warp >= kMmaWarp) {  // the item warps look for their first item before they join
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    tmem = *s_tmem;
  }
  int n_issued = 0;               // the loader's tiles

  if (warp < C::kSoftWarps) {
    // ================================================================ softmax
    const int grp = warp >> 2, w4 = warp & 3, row = tid & 127;  // rows grp * kRows ..; TMEM lane (key of a tile)
    float* red = s_red + grp * 4 * kRows;
    int* fail = s_fail + grp * 4;
    bool failed = false, stop = false;
    int g = 0;  // tiles so far, over all items
    for (int n = 0; !stop; ++n) {
      const Item<R>& it = items[n % C::kItems];
      if (!wait_all(bar_ready + n % C::kItems, (n / C::kItems) & 1, abort_flag, 3)) failed = true;
      if (softmax_bar_or(grp, failed || *abort_flag)) {
        *abort_flag = 1;
        break;
      }
      const int n_t = it.n_t, kn = it.kn;
      if (n_t < 0) break;
      const int lim_min = it.lim_min;
      const bool idle = grp > 0 && it.o_row[grp * kRows] < 0;  // no row of the group is real: it only keeps step
      // Rows in pairs (packed fp32 arithmetic).  nm: the reference (base 2),
      // negated, 0 until the item's first tile sets it (every row that sees a
      // key sees the split's first one); seen: bit r once row r's is set.
      constexpr int kPairs = kRows / 2;
      float2 nm[kPairs], l[kPairs], qm[kPairs];
      uint32_t seen = 0u;
#pragma unroll
      for (int r = 0; r < kPairs; ++r) {
        nm[r] = l[r] = make_float2(0.f, 0.f);
        qm[r] = make_float2(it.qm[grp * kRows + 2 * r], it.qm[grp * kRows + 2 * r + 1]);
      }
      for (int t = 0; t < n_t; ++t, ++g) {
        const int buf = g & 1, s = g % C::kStages;
        const int key = t * kTile + row;
        const bool live = key < kn;
        const float ks = live ? it.ks[key >> 6] : 0.f, wv = live ? it.vs[key >> 6] : 0.f;
        const float lift = log2_up(wv);  // what the key's scale adds to its score, as the reference sees it
        if (!wait_all(bar_s + buf, (g >> 1) & 1, abort_flag, 4)) failed = true;
        if (idle) {
          // (its columns of P and O^T are not looked at)
          if (g >= 2 && !wait_all(bar_of + buf, ((g - 2) >> 1) & 1, abort_flag, 6)) failed = true;
          if (lane == 0) mbar_arrive(bar_p + buf);
          continue;  // also where a wait gave up: the group's warps leave together, at the next item
        }
        tc_fence_after();
        constexpr int kLd = (3 * kRows + 7) / 8 * 8;
        uint32_t u[kLd];
        tmem_ld_row<kLd>(tmem + (static_cast<uint32_t>(w4 * 32) << 16) + buf * kN + grp * 3 * kRows, u);
        tc_fence_before();
        const bool edge = (t + 1) * kTile > lim_min;  // uniform: some row does not see the whole tile
        uint32_t hidden = 0u;  // rows that do not see this thread's key
        if (edge) {
#pragma unroll
          for (int r = 0; r < kRows; ++r) hidden |= (key >= it.lim[grp * kRows + r] ? 1u : 0u) << r;
        }
        float2 x[kPairs];  // scores in base 2, less the reference
        bool big = false;
        const float2 ks2 = make_float2(ks, ks);
#pragma unroll
        for (int r = 0; r < kPairs; ++r) {
          auto at = [&](int k) {
            return make_float2(__uint_as_float(u[k * kRows + 2 * r]), __uint_as_float(u[k * kRows + 2 * r + 1]));
          };
          x[r] = ffma2(fadd2(fadd2(at(0), at(1)), at(2)), fmul2(qm[r], ks2), nm[r]);
          big = big || fmaxf(x[r].x, x[r].y) + lift > kMoveLog2;  // (masked keys can only ask for the look below)
        }
        float al[kRows];
#pragma unroll
        for (int r = 0; r < kRows; ++r) al[r] = 1.f;
        if (t == 0 || softmax_bar_or(grp, big || failed || *abort_flag)) {
          // the first tile sets the references; some row's may have to move (or a wait gave up)
          float top[kRows];
#pragma unroll
          for (int r = 0; r < kRows; ++r)
            top[r] = (hidden >> r) & 1u ? -INFINITY : (r & 1 ? x[r / 2].y : x[r / 2].x) + lift;  // NaN scores show in p
          const float mine = warp_max_rows(top);
          if (lane % (32 / kRows) == 0) red[w4 * kRows + lane / (32 / kRows)] = mine;
          if (lane == 0) fail[w4] = failed || *abort_flag;
          softmax_bar(grp);
          if (fail[0] | fail[1] | fail[2] | fail[3]) {
            *abort_flag = 1;
            stop = true;
            break;
          }
#pragma unroll
          for (int r = 0; r < kRows; ++r) top[r] = -INFINITY;
#pragma unroll
          for (int i = 0; i < kRows; ++i) {  // four rows of a warp a load
            const float4 v = reinterpret_cast<const float4*>(red)[i];
            const int r = 4 * i % kRows;
            top[r] = fmaxf(top[r], v.x);
            top[r + 1] = fmaxf(top[r + 1], v.y);
            top[r + 2] = fmaxf(top[r + 2], v.z);
            top[r + 3] = fmaxf(top[r + 3], v.w);
          }
#pragma unroll
          for (int r = 0; r < kRows; ++r) {
            const float mx = top[r];
            const bool first = !((seen >> r) & 1u);
            if (mx > (first ? -INFINITY : kMoveLog2)) {
              float& mr = r & 1 ? nm[r / 2].y : nm[r / 2].x;
              float& lr = r & 1 ? l[r / 2].y : l[r / 2].x;
              float& xr = r & 1 ? x[r / 2].y : x[r / 2].x;
              al[r] = first ? 0.f : ex2_approx(-mx);
              lr *= al[r];
              mr -= mx;
              xr -= mx;
              seen |= 1u << r;
            }
          }
        }
        // P and alpha of this buffer are free once tile g-2 is added up
        if (g >= 2 && !wait_all(bar_of + buf, ((g - 2) >> 1) & 1, abort_flag, 6)) failed = true;
        // Rows of V past the sequence may hold anything: they are cleared, so
        // that a weight of 0 adds exactly nothing.  In a row that only some of
        // the new tokens see each NaN is cleared, and its dim noted with the
        // first key for the output warps, who give it to the rows that see it.
        // Group 0 does so (the MMA waits for every group).
        if (edge && grp == 0) {
          // long done: S needed it
          if (!wait_all(bar_full + s, (g / C::kStages) & 1, abort_flag, 5)) failed = true;
          const uint32_t vrow = smem_u32(smem + s * C::kStage + C::kOffV);
          if (!live) {
#pragma unroll
            for (int c = 0; c < D; c += 16) st_shared_v4(vrow + swizzled<D>(row, c), 0u, 0u, 0u, 0u);
          } else if (key >= lim_min) {
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
              const uint4 v = ld_shared_v4(vrow + swizzled<D>(row, c));
              uint32_t w[4] = {v.x, v.y, v.z, v.w}, nan = 0u;
#pragma unroll
              for (int i = 0; i < 4; ++i) nan |= (w[i] & 0x7f7f7f7fu) + 0x01010101u;
              if (nan & 0x80808080u) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  for (int k = 0; k < 4; ++k) {
                    if (((w[i] >> (8 * k)) & 0x7fu) != 0x7fu) continue;
                    atomicMin(s_nan + buf * D + c + 4 * i + k, key);
                    w[i] &= ~(0xffu << (8 * k));
                  }
                }
                st_shared_v4(vrow + swizzled<D>(row, c), w[0], w[1], w[2], w[3]);
              }
            }
          }
        }
        const float2 wv2 = make_float2(wv, wv);
        uint32_t code[3][kPairs];  // two rows each
#pragma unroll
        for (int r = 0; r < kPairs; ++r) {
          float2 pr = make_float2(ex2_approx(x[r].x), ex2_approx(x[r].y));
          if (edge) {
            if ((hidden >> (2 * r)) & 1u) pr.x = 0.f;
            if ((hidden >> (2 * r + 1)) & 1u) pr.y = 0.f;
          }
          l[r] = fadd2(l[r], pr);
          float2 w = fmul2(pr, wv2);
#pragma unroll
          for (int k = 0; k < 3; ++k) {
            const float2 tm = k < 2 ? make_float2(lead3(w.x), lead3(w.y)) : w;
            code[k][r] = e5m2x2(tm.x, tm.y);
            if (k < 2) w = fadd2(w, make_float2(-tm.x, -tm.y));
          }
        }
#pragma unroll
        for (int k = 0; k < 3; ++k) {  // a term's rows lie together
          const uint32_t at = sP + buf * kN * kTile + p_at((grp * 3 + k) * kRows, row);
          const uint32_t lo = code[k][0] | (code[k][1] << 16);
          if constexpr (kRows == 8)
            asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(at), "r"(lo),
                         "r"(code[k][2] | (code[k][3] << 16))
                         : "memory");
          else
            asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(lo) : "memory");
        }
        if (row < kRows) {
          float v = 1.f;
#pragma unroll
          for (int r = 0; r < kRows; ++r)
            if (row == r) v = al[r];
          s_alpha[buf * R + grp * kRows + row] = v;
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
      for (int r = 0; r < kRows; ++r) {
        const float lr = warp_sum(r & 1 ? l[r / 2].y : l[r / 2].x);
        if (lane == 0) ml[(1 + w4) * R + grp * kRows + r] = lr;
        if (row == 0) ml[grp * kRows + r] = r & 1 ? -nm[r / 2].y : -nm[r / 2].x;
      }
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar_ml + (n & 1));
        mbar_arrive(bar_free + n % C::kItems);
      }
    }
  } else if (warp < kItemWarp) {
    // ================================================================ output
    const int dd = tid - 32 * kOut0;
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
        constexpr int kLd = (3 * kRows + 7) / 8 * 8;
        const uint32_t o_at = tmem + (static_cast<uint32_t>((warp - kOut0) * 32) << 16) + (2 + buf) * kN;
#pragma unroll
        for (int q = 0; q < C::kGroups; ++q) {
          uint32_t u[kLd];
          tmem_ld_row<kLd>(o_at + q * 3 * kRows, u);
#pragma unroll
          for (int r = 0; r < kRows; ++r)
            acc[q * kRows + r] =
                fmaf(acc[q * kRows + r], s_alpha[buf * R + q * kRows + r],
                     __uint_as_float(u[r]) + __uint_as_float(u[kRows + r]) + __uint_as_float(u[2 * kRows + r]));
        }
        tc_fence_before();
        if ((t + 1) * kTile > it.lim_min && it.lim_min < it.kn) {  // NaN values that some rows see
          const int first = s_nan[buf * D + dd];
          if (first != kNoKey) {
#pragma unroll
            for (int r = 0; r < R; ++r)
              if (first < it.lim[r]) acc[r] = NAN;
            s_nan[buf * D + dd] = kNoKey;
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_of + buf);
      }
      if (!ok || !wait_all(bar_ml + (n & 1), (n >> 1) & 1, abort_flag, 11)) break;
      const float* ml = s_ml + (n & 1) * 5 * R;
      const int split = it.split;
      const bool direct = it.direct != 0;
      const float vref = it.vref;
      // Lane r forms row r's factor and LSE (every lane all of them took 3.5 us
      // for 24 rows); what the slot holds is read before it is given back.
      // l is 0 exactly where the row sees no key of the split (NaN, not 0, where a score is NaN).
      int o_row = -1, lse_row = -1;
      float lr = 0.f, lse = -INFINITY;
      if (lane < R) {
        lr = (ml[R + lane] + ml[2 * R + lane]) + (ml[3 * R + lane] + ml[4 * R + lane]);
        if (lr != 0.f) lse = (ml[lane] + __log2f(lr)) * 0.6931471805599453f;
        o_row = it.o_row[lane];
        lse_row = it.lse_row[lane];
      }
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar_mf + (n & 1));
        mbar_arrive(bar_free + n % C::kItems);
      }
      const float inv = lr == 0.f ? 0.f : (1.f / kWeightScale) / lr;
      const unsigned none = __ballot_sync(0xffffffffu, lr == 0.f);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        acc[r] = acc[r] * __shfl_sync(0xffffffffu, inv, r) * vref;
        if ((none >> r) & 1u) acc[r] = 0.f;
      }
      if (p.cluster != 0) {
        // over the stages, whose last tile has been multiplied
#pragma unroll
        for (int r = 0; r < R; ++r) s_part[r * D + dd] = acc[r];
        if (dd < R) {
          s_part_lse[dd] = lse;
          s_part_row[dd] = o_row;
          s_part_row[R + dd] = lse_row;
        }
        continue;
      }
      if (dd < R && o_row >= 0) {
        if (direct)
          p.lse[lse_row] = lse;
        else
          p.lse_part[static_cast<long long>(o_row) * p.n_split + split] = lse;
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int to = __shfl_sync(0xffffffffu, o_row, r);
        if (to < 0) break;  // rows are in order, those past the last behind
        if (direct)
          static_cast<__nv_bfloat16*>(p.o)[static_cast<long long>(to) * D + dd] = __float2bfloat16_rn(acc[r]);
        else
          p.o_part[(static_cast<long long>(to) * p.n_split + split) * D + dd] = acc[r];
      }
    }
  } else if (warp < kMmaWarp) {
    // ================================================================ items
    // Every item warp finds every item; the first one writes its description
    // and tells the loader, each one turns its own rows of q into e5m2 terms.
    // Item i of the whole call: j = i / H counts (sequence, split) pairs, the
    // full splits of all sequences first and the shorter last ones after them,
    // i % H is the KV head and block of its rows (so neighbouring CTAs read
    // the same cache rows).  The lanes hold 32 sequences at a time; j only
    // grows, so they walk the batch once for the full splits and once for the
    // rest.
    const int n_rblk = static_cast<int>(p.n_rblk.d), H = static_cast<int>(p.H.d), G = static_cast<int>(p.G.d);
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
    // kLanes lanes share a row of q, each a run of kDims of it; kPasses times
    // kPassRows rows.  One pass of q is loaded an item ahead; two would not fit
    // the registers.
    constexpr int kPg = C::kMaxBlocks / 32, kLanes = R == 4 ? 8 : 4, kDims = D / kLanes;
    constexpr int kPassRows = C::kItemWarps * 32 / kLanes, kPasses = (R + kPassRows - 1) / kPassRows;
    constexpr bool kAhead = kPasses == 1;
    const bool leads = warp == kItemWarp;
    const int qr = ((warp - kItemWarp) * 32 + lane) / kLanes, qd = lane % kLanes * kDims;
    // row r of an item: its place, and this lane's part of its q
    auto row_of = [&](int hkv, int row0, int r, int& tok, int& hq) {
      const int row = row0 + r;
      tok = p.G.div(row);
      hq = hkv * G + row - tok * G;
      return row < rows;
    };
    auto load_q = [&](int b, int tok, int hq, bool real, uint4 (&q)[kDims / 8]) {
      const __nv_bfloat16* at =
          static_cast<const __nv_bfloat16*>(p.q) + ((static_cast<long long>(b) * p.Nq + tok) * p.Hq + hq) * D + qd;
#pragma unroll
      for (int c = 0; c < kDims / 8; ++c)
        q[c] = real ? *reinterpret_cast<const uint4*>(at + 8 * c) : make_uint4(0u, 0u, 0u, 0u);
    };
    struct Found {  // an item found, its page numbers on their way
      bool more;
      int b, split, len, hkv, row0;
      int pg[kPg];
    };
    struct Loading {  // its scales and q on their way
      bool more;
      int k0, kn, n_blk, len, b, hkv, row0;
      float ks[kPg], vs[kPg];
      uint4 q[kAhead ? kDims / 8 : 1];
    };
    // Clustered: one item a CTA, split by rank, nothing to look for (empty
    // splits are items too: the cluster's combine wants them all).
    bool more = p.cluster ? true : next_block();
    unsigned item = blockIdx.x;
    auto find = [&]() {
      Found f;
      if (p.cluster) {
        const unsigned g = blockIdx.x / p.cluster, h = p.H.div(g) * p.H.d;
        f.more = item == blockIdx.x;
        item += gridDim.x;
        f.b = p.H.div(g);
        f.hkv = p.n_rblk.div(g - h);
        f.row0 = (static_cast<int>(g - h) - f.hkv * n_rblk) * R;
        f.split = blockIdx.x % p.cluster;
        f.len = p.seqlens[f.b];
        if (f.len < 0 || f.len > p.max_seqlen) {
          record(1, kDevBadSeqlen);
          f.len = f.len < 0 ? 0 : p.max_seqlen;
        }
        const int k0 = f.split * p.chunk, n_blk = f.more ? (min(p.chunk, f.len - k0) + 63) / 64 : 0;
#pragma unroll
        for (int k = 0; k < kPg; ++k) {
          const int blk = 32 * k + lane;
          f.pg[k] = leads && blk < n_blk
                        ? p.block_table[static_cast<long long>(f.b) * p.max_blocks + p.page.div(k0 + 64 * blk)]
                        : 0;
        }
        return f;
      }
      const unsigned j = p.H.div(item), h = item - j * H;
      item += gridDim.x;  // fits: the host sees to it
      while (more && j >= before + total) {
        more = next_block();
        if (!more && full_phase) {
          full_phase = false;
          b0 = -32;
          total = 0;
          more = next_block();
        }
      }
      f.more = more;
      f.b = f.split = f.len = 0;
      f.hkv = p.n_rblk.div(h);
      f.row0 = (h - f.hkv * n_rblk) * R;
#pragma unroll
      for (int k = 0; k < kPg; ++k) f.pg[k] = 0;
      if (more) {
        const int rel = static_cast<int>(j - before);
        const unsigned who = __ballot_sync(0xffffffffu, cnt > 0 && rel >= excl && rel < excl + cnt);
        const int src = __ffs(who) - 1;
        f.b = b0 + src;
        f.len = __shfl_sync(0xffffffffu, Lb, src);
        f.split = full_phase ? rel - __shfl_sync(0xffffffffu, excl, src) : p.split.div(f.len);
        const int k0 = f.split * p.chunk, n_blk = (min(p.chunk, f.len - k0) + 63) / 64;
#pragma unroll
        for (int k = 0; k < kPg; ++k) {
          const int blk = 32 * k + lane;
          if (leads && blk < n_blk)
            f.pg[k] = p.block_table[static_cast<long long>(f.b) * p.max_blocks + p.page.div(k0 + 64 * blk)];
        }
      }
      return f;
    };
    // Item n, found: tells the loader, starts its other loads (before the
    // loader's, behind which they would wait).  False: a wait gave up.
    bool ok = true;
    auto open = [&](Found& f, int n) {
      Loading a;
      const int slot = n % C::kItems;
      Item<R>& it = items[slot];
      a.more = f.more;
      a.k0 = f.split * p.chunk;
      a.kn = max(0, min(p.chunk, f.len - a.k0));
      a.n_blk = (a.kn + 63) / 64;
      a.len = f.len;
      a.b = f.b;
      a.hkv = f.hkv;
      a.row0 = f.row0;
      if (f.more) {
#pragma unroll
        for (int k = 0; k < kPg; ++k) {
          if (f.pg[k] < 0 || f.pg[k] >= p.num_pages) {
            record(2, kDevBadPage);
            f.pg[k] = 0;  // keep every load inside the page pool; the result is flagged
          }
          a.ks[k] = a.vs[k] = 0.f;
          if (leads && 32 * k + lane < a.n_blk) {
            a.ks[k] = p.k_scales[static_cast<long long>(f.pg[k]) * p.Hkv + f.hkv];
            a.vs[k] = p.v_scales[static_cast<long long>(f.pg[k]) * p.Hkv + f.hkv];
          }
        }
        if constexpr (kAhead) {
          int tok, hq;
          const bool real = row_of(f.hkv, f.row0, qr, tok, hq);
          load_q(f.b, tok, hq, real, a.q);
        }
      }
      if (n >= C::kItems && !wait_all(bar_free + slot, (n / C::kItems - 1) & 1, abort_flag, 12)) {
        ok = false;
        return a;
      }
      if (!leads) return a;
      if (lane == 0) {
        it.n_t = f.more ? (a.kn + kTile - 1) / kTile : -1;
        it.kn = a.kn;
        it.split = f.split;
        it.hkv = f.hkv;
        it.lim_min = min(a.kn, f.len - p.Nq + 1 + static_cast<int>(p.G.div(f.row0)) - a.k0);
        it.direct = f.len <= p.chunk;
      }
      if (f.more) {
#pragma unroll
        for (int k = 0; k < kPg; ++k)
          if (32 * k + lane < a.n_blk) it.page[32 * k + lane] = f.pg[k];
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_pages + slot);
      return a;
    };
    // Item n, its loads landed: the rest of its description, and its Q operand.
    auto finish = [&](const Loading& cur, int n) {
      const int slot = n % C::kItems;
      Item<R>& it = items[slot];
      if (cur.more) {
        // q as three e5m2 terms a row
        const uint32_t q_at = sQ + slot * C::kQBytes;
#pragma unroll
        for (int ps = 0; ps < kPasses; ++ps) {
          const int r = ps * kPassRows + qr;
          if (R % kPassRows != 0 && r >= R) break;  // uniform: whole warps
          int tok, hq;
          const bool real = row_of(cur.hkv, cur.row0, r, tok, hq);
          uint4 q[kDims / 8];
          if constexpr (kAhead) {
#pragma unroll
            for (int c = 0; c < kDims / 8; ++c) q[c] = cur.q[c];
          } else {
            load_q(cur.b, tok, hq, real, q);
          }
          uint32_t amax = 0u;
#pragma unroll
          for (int c = 0; c < kDims / 8; ++c) {
            const uint32_t w[4] = {q[c].x, q[c].y, q[c].z, q[c].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) amax = max(amax, max((w[k] << 16) & 0x7fffffffu, w[k] & 0x7fff0000u));
          }
#pragma unroll
          for (int o = kLanes / 2; o > 0; o >>= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, o));
          const bool fin = amax < 0x7f800000u;  // bits of the row's largest magnitude
          const int e = fin ? max(static_cast<int>(amax >> 23) - 127, -100) : 0;
          const float f = __uint_as_float(static_cast<uint32_t>(14 - e + 127) << 23);
#pragma unroll
          for (int c = 0; c < kDims / 8; ++c) {  // 8 values: 8 bytes a term, at a multiple of 8
            const uint32_t w[4] = {q[c].x, q[c].y, q[c].z, q[c].w};
            float x[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              x[2 * i] = bf16lo(w[i]) * f;
              x[2 * i + 1] = bf16hi(w[i]) * f;
            }
#pragma unroll
            for (int k = 0; k < 3; ++k) {
              float t3[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                t3[i] = lead3(x[i]);
                x[i] -= t3[i];
              }
              const uint32_t at = q_at + swizzled<D>(column<R, kRows>(k, r), qd + 8 * c);
              asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(at),
                           "r"(e5m2x2(t3[0], t3[1]) | (e5m2x2(t3[2], t3[3]) << 16)),
                           "r"(e5m2x2(t3[4], t3[5]) | (e5m2x2(t3[6], t3[7]) << 16))
                           : "memory");
            }
          }
          if (lane % kLanes == 0) {
            it.lim[r] = min(cur.kn, cur.len - p.Nq + 1 + tok - cur.k0);
            it.o_row[r] = real ? (cur.b * p.Nq + tok) * p.Hq + hq : -1;
            it.lse_row[r] = (cur.b * p.Hq + hq) * p.Nq + tok;
            // a row with an infinity or NaN: every score NaN
            it.qm[r] = fin ? __uint_as_float(static_cast<uint32_t>(e - 14 + 127) << 23) * p.scale_log2 : NAN;
          }
        }
        if (leads) {
          float vref = 0.f;
#pragma unroll
          for (int k = 0; k < kPg; ++k) vref = fmaxf(vref, cur.vs[k]);
          vref = warp_max(vref);
#pragma unroll
          for (int k = 0; k < kPg; ++k) {
            if (32 * k + lane < cur.n_blk) {
              it.ks[32 * k + lane] = cur.ks[k];
              // at most kWeightScale, however small the scales are
              it.vs[32 * k + lane] = vref > 0.f ? cur.vs[k] / vref * kWeightScale : 0.f;
            }
          }
          if (lane == 0) it.vref = vref;
        }
        fence_proxy_async_smem();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_ready + slot);
    };
    Found nxt = find();
    __syncthreads();
    // the first item by itself, then with item n+1's loads and item n+2's page
    // numbers on their way while item n is finished
    Loading cur = open(nxt, 0);
    if (cur.more) nxt = find();
    finish(cur, 0);
    if (cur.more) {
      cur = open(nxt, 1);
      if (cur.more) nxt = find();
      for (int n = 1; ok; ++n) {
        Loading then;
        then.more = false;
        if (cur.more) {
          then = open(nxt, n + 1);
          if (!ok) break;
          if (then.more) nxt = find();
        }
        finish(cur, n);
        if (!cur.more) break;
        cur = then;
      }
    }
  } else if (warp == kMmaWarp) {
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
          mma_f8_ss(tmem + (2 + (g & 1)) * kN, desc(v + c * D, C::kTileBytes),
                    sdesc_sw0(pb + p_at(0, c), 128, 16 * kTile), idesc_o, c > 0);
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
            const int blk = 2 * t + i, key = k0 + 64 * blk, page = it.page[blk];
            const int row = key - static_cast<int>(p.page.div(key)) * p.page_size;
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
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmem);
  }
  if (p.cluster == 0) return;
  if (*abort_flag) {  // there may be no result: this CTA writes none (the others' are as undefined, and reported)
    for (int r = tid; r < R; r += C::kThreads) s_part_row[r] = -1;
    __syncthreads();
  }
  // Combine within the cluster, through the CTAs' shared memory: rank k takes
  // rows k, k + cluster, ...  The arithmetic, in its order, is the combine
  // kernel's (which has at most one split a sum for so few), so the same
  // splits give the same bits either way.
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
  auto peer = [](const void* at, int rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(at)), "r"(rank));
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
  };
  for (int i = tid; i < R * D; i += C::kThreads) {
    const int r = i / D, dd = i % D;
    if (r % p.cluster != static_cast<int>(blockIdx.x % p.cluster) || s_part_row[r] < 0) continue;
    float lv[8], mx = -INFINITY;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      lv[k] = k < p.n_split ? peer(s_part_lse + r, k) : -INFINITY;
      mx = fmaxf(mx, lv[k]);
    }
    if (mx == -INFINITY) mx = 0.f;
    float a = 0.f, sum = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float w = expf(lv[k] - mx);
      sum = __fadd_rn(sum, w);
      a = __fadd_rn(a, __fmul_rn(w, k < p.n_split ? peer(s_part + i, k) : 0.f));
    }
    const bool none = sum == 0.f;
    static_cast<__nv_bfloat16*>(p.o)[static_cast<long long>(s_part_row[r]) * D + dd] =
        __float2bfloat16_rn(none ? 0.f : a / sum);
    if (dd == 0) p.lse[s_part_row[R + r]] = none ? -INFINITY : mx + logf(sum);
  }
  // the others may still read this CTA's shared memory
  asm volatile("barrier.cluster.arrive;\n\tbarrier.cluster.wait;" ::: "memory");
}

// LSE = ln sum_s exp(LSE_s), O = sum_s exp(LSE_s - LSE) O_s for each row of q.
// A block of kWarps warps takes kCols columns of a row, a warp every
// kWarps-th split, kBatch splits' loads in flight.  Whatever the form, 32 sums
// are kept, of the splits s, s + 32, ... each, and then added in order: a row's
// bits depend on its own splits alone, not on the form that other rows or the
// table's width ask for.  Many rows, or few splits: eight warps and the whole
// row; with at most eight splits these have a sum each and the other 24 are left
// out (1728 rows of up to 5 splits: the step takes 31.4 us so, 32.0 with all).
// Few rows of many splits (a few long sequences): 32 warps for each 32
// columns, as one block's loads are then what the step waits for (64 rows of
// 512 splits: 39 us in whole rows by eight warps, 5 us so; 512 rows of 32
// splits: 3 us and 30 us).
template <int D, int kCols, int kWarps, int kBatch>
__global__ void __launch_bounds__(32 * kWarps) decode_fp8_combine_kernel(const DecodeFp8CombineParams p) {
  constexpr int kV = kCols / 32, kBlocks = D / kCols;
  constexpr int kSums = kBatch == 1 ? 1 : 32 / kWarps, kAll = kSums * kWarps;  // of a warp, of the block
  static_assert(kBatch % kSums == 0, "split s of a batch belongs to sum s % 32");
  __shared__ float s_max[kWarps], s_tot[kAll];
  __shared__ float s_acc[kAll][kCols];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int qrow = blockIdx.x / kBlocks, col0 = blockIdx.x % kBlocks * kCols;
  const int bi = qrow / p.Hq, hq = qrow - bi * p.Hq, b = bi / p.Nq, i = bi - b * p.Nq;
  grid_release();
  // launched as a programmatic dependent of the split kernel: wait until all
  // of its partials are written and visible
  grid_wait();
  int Lb = p.seqlens[b];
  Lb = Lb < 0 ? 0 : (Lb > p.max_seqlen ? p.max_seqlen : Lb);
  const int ns = (Lb + p.chunk - 1) / p.chunk;
  if (ns == 1) return;  // written by the split kernel
  const float* lp = p.lse_part + static_cast<long long>(qrow) * p.n_split;
  const float* op = p.o_part + static_cast<long long>(qrow) * p.n_split * D + col0 + kV * lane;
  // kBatch splits of the warp: their LSEs and this lane's columns.  The first
  // batch is loaded before the largest LSE is known.
  float lv[kBatch], ov[kBatch][kV];
  auto load = [&](int s) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int su = s + u * kWarps;
      lv[u] = su < ns ? lp[su] : -INFINITY;
#pragma unroll
      for (int k = 0; k < kV; ++k) ov[u][k] = 0.f;
      if (su < ns) {
        const float* o = op + static_cast<long long>(su) * D;
        if (kV == 4) {
          const float4 v = *reinterpret_cast<const float4*>(o);
          ov[u][0] = v.x; ov[u][1 % kV] = v.y; ov[u][2 % kV] = v.z; ov[u][3 % kV] = v.w;
        } else if (kV == 2) {
          const float2 v = *reinterpret_cast<const float2*>(o);
          ov[u][0] = v.x; ov[u][1 % kV] = v.y;
        } else {
          ov[u][0] = *o;
        }
      }
    }
  };
  load(warp);
  float mx = -INFINITY;
  for (int s = threadIdx.x; s < ns; s += 32 * kWarps) mx = fmaxf(mx, lp[s]);
  mx = warp_max(mx);
  if (lane == 0) s_max[warp] = mx;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, s_max[w]);
  if (mx == -INFINITY) mx = 0.f;  // no key seen (or every LSE NaN): the weights are then 0 (NaN)
  float tot[kSums], acc[kSums][kV];
#pragma unroll
  for (int i = 0; i < kSums; ++i) {
    tot[i] = 0.f;
#pragma unroll
    for (int k = 0; k < kV; ++k) acc[i][k] = 0.f;
  }
  for (int s = warp; s < ns; s += kBatch * kWarps) {
    if (s != warp) load(s);
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const float w = expf(lv[u] - mx);
      tot[u % kSums] += w;
#pragma unroll
      for (int k = 0; k < kV; ++k) acc[u % kSums][k] = fmaf(w, ov[u][k], acc[u % kSums][k]);
    }
  }
#pragma unroll
  for (int i = 0; i < kSums; ++i) {
    if (warp + i * kWarps >= ns) break;  // (0, not read)
    if (lane == 0) s_tot[warp + i * kWarps] = tot[i];
#pragma unroll
    for (int k = 0; k < kV; ++k) s_acc[warp + i * kWarps][kV * lane + k] = acc[i][k];
  }
  __syncthreads();
  if (threadIdx.x >= kCols) return;
  float a = 0.f, sum = 0.f;
  for (int i0 = 0; i0 < min(ns, kAll); i0 += 8) {  // the sums past the last split are 0
    float av[8], tv[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      av[i] = i0 + i < ns ? s_acc[i0 + i][threadIdx.x] : 0.f;
      tv[i] = i0 + i < ns ? s_tot[i0 + i] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      a += av[i];
      sum += tv[i];
    }
  }
  const bool none = sum == 0.f;
  static_cast<__nv_bfloat16*>(p.o)[static_cast<long long>(qrow) * D + col0 + threadIdx.x] =
      __float2bfloat16_rn(none ? 0.f : a / sum);
  if (threadIdx.x == 0 && col0 == 0)
    p.lse[(static_cast<long long>(b) * p.Hq + hq) * p.Nq + i] = none ? -INFINITY : mx + logf(sum);
}

template <int D, int R>
cudaError_t launch_rows(DecodeFp8Params p, int dev, int sms, cudaStream_t stream) {
  using C = Cfg<D, R>;
  auto kern = decode_fp8_split_kernel<D, R>;
  // asked for once a device (bit dev of `set`; past 63 every time)
  static std::atomic<unsigned long long> set{0};
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
  cudaError_t e = cudaSuccess;
  if (!(set.load(std::memory_order_acquire) & bit) || bit == 0ull) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kAlloc);
    if (e != cudaSuccess) return e;
    set.fetch_or(bit, std::memory_order_release);
  }
  const int rows = p.Nq * (p.Hq / p.Hkv);
  // the most items there can be: the lengths are known on the device alone
  const long long items = static_cast<long long>(p.Hkv) * ((rows + R - 1) / R) * p.B * p.n_split;
  const long long ctas = static_cast<long long>(sms) * C::kCtas;
  p.rows = rows;
  p.n_rblk = FastDiv((rows + R - 1) / R);
  p.H = FastDiv(p.Hkv * ((rows + R - 1) / R));
  p.G = FastDiv(p.Hq / p.Hkv);
  p.page = FastDiv(p.page_size);
  p.split = FastDiv(p.chunk);
  // Few splits and few of them in all: the splits of a group of rows form a
  // cluster, which combines them itself; no more CTAs than places for them.
  int cluster = 1;
  while (cluster < p.n_split) cluster *= 2;
  const long long clustered = items / p.n_split * cluster;
  if (p.n_split > 1 && cluster <= 8 && clustered <= ctas) {
    p.cluster = cluster;
    return launch_dependent_clusters(kern, dim3(static_cast<unsigned>(clustered)), cluster, C::kThreads, C::kAlloc,
                                     stream, p);
  }
  p.cluster = 0;
  e = launch_dependent(kern, dim3(static_cast<unsigned>(items < ctas ? items : ctas)), C::kThreads, C::kAlloc, stream, p);
  if (e != cudaSuccess || p.n_split == 1) return e;
  const DecodeFp8CombineParams c = {p.o_part, p.lse_part, p.seqlens, p.o, p.lse, p.Nq, p.Hq, p.max_seqlen, p.chunk,
                                    p.n_split};
  const unsigned q_rows = static_cast<unsigned>(p.B) * p.Nq * p.Hq;
  if (p.n_split <= 8) return launch_dependent(decode_fp8_combine_kernel<D, D, 8, 1>, dim3(q_rows), 256, 0, stream, c);
  if (q_rows >= 2u * sms || p.n_split <= 32)
    return launch_dependent(decode_fp8_combine_kernel<D, D, 8, 4>, dim3(q_rows), 256, 0, stream, c);
  return launch_dependent(decode_fp8_combine_kernel<D, 32, 32, 8>, dim3(q_rows * (D / 32)), 1024, 0, stream, c);
}

template <int D>
cudaError_t launch_d(const DecodeFp8Params& p, cudaStream_t stream) {
  int dev, sms;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int rows = p.Nq * (p.Hq / p.Hkv);
  if (rows <= 4) return launch_rows<D, 4>(p, dev, sms, stream);
  if (rows <= 8) return launch_rows<D, 8>(p, dev, sms, stream);
  // blocks of 16 or 24 rows: whichever reads the cache fewer times, 16 where equal
  if ((rows + 23) / 24 < (rows + 15) / 16) return launch_rows<D, 24>(p, dev, sms, stream);
  return launch_rows<D, 16>(p, dev, sms, stream);
}

}  // namespace

cudaError_t launch_decode_fp8(const DecodeFp8Params& p, cudaStream_t stream) {
  return p.d == 64 ? launch_d<64>(p, stream) : launch_d<128>(p, stream);
}

cudaError_t status_word_decode_fp8(uint32_t** at) { return cudaGetSymbolAddress(reinterpret_cast<void**>(at), g_decode_fp8_status); }

}  // namespace attn

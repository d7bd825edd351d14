// Which blocks of a paged cache a query attends to, for sm_103a: bounds of
// the keys of each 64-key block, the scores that they allow, and the choice of
// the largest ones.
//
// Bounds: lo_i = min, hi_i = max over the block's keys of channel i; exact in
// bf16, whatever the order of the keys.
//
// Score of block j for a query row of one KV head, with q+ = max(q, 0) and
// q- = min(q, 0) for each of the group's heads:
//     score(j) = max over heads of sum_i (q+_i hi_ij + q-_i lo_ij),
// no key of the block has a larger <q, k>.
//
// Choice: the row's first `sink` and last `local` blocks, then the largest
// scores, the lower index first among equals; the order is that of the scores
// in 64 bits.  The scores are formed in fp32 first, off by at most E, so a block
// is in where its score is above the k-th largest T by more than 2 E, out where
// it is that far below, and only the few in between are scored again in 64 bits.
// An fp32 sum of 256 terms, truncated at worst at each addition, is off by at
// most 2^-15 of the sum of magnitudes, and that is at most |q| max_j |m_j| with
// m = max(|lo|, |hi|) (Cauchy and Schwarz).  Where a norm cannot be told in fp32
// there is no E, and all blocks are scored again.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "launch.h"
#include "ptx.cuh"
#include "rope.cuh"

namespace attn {
namespace {

__device__ uint32_t g_select_status;

__device__ __forceinline__ void record(uint32_t site, uint32_t code) {
  atomicCAS(&g_select_status, 0u, (site << 8) | code);
}

constexpr int kThreads = 256;
constexpr uint64_t kWaitLimitNs = 2000000000ull;  // 2 s: no legitimate wait comes close
constexpr int kBlock = kSelectBlock;  // keys of a block

__device__ __forceinline__ int clamped_len(const int* seqlens, int b, int cap, bool report) {
  const int len = seqlens[b];
  if (report && (len < 0 || len > cap)) record(1, kDevBadSeqlen);
  return min(max(len, 0), cap);
}

// ---------------------------------------------------------------------------
// Bounds.  One CTA for each touched block and 64 chunks of 8 channels: four
// groups of 64 threads take 16 rows each, a thread's loads all in flight at
// once, and meet in shared memory.  Bound by memory: each key read once (prompts of
// 8191 tokens padded, 104 MB: 21 us, 5 TB/s; a step's new tokens: 3.2 us, latency).
__device__ __forceinline__ uint32_t min_nan2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t max_nan2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint4 min4(const uint4& a, const uint4& b) {
  return make_uint4(min_nan2(a.x, b.x), min_nan2(a.y, b.y), min_nan2(a.z, b.z), min_nan2(a.w, b.w));
}
__device__ __forceinline__ uint4 max4(const uint4& a, const uint4& b) {
  return make_uint4(max_nan2(a.x, b.x), max_nan2(a.y, b.y), max_nan2(a.z, b.z), max_nan2(a.w, b.w));
}

__global__ void __launch_bounds__(kThreads) bounds_kernel(const KeyBoundsParams p, int slabs) {
  grid_depends();
  __shared__ uint4 s_lo[3][64], s_hi[3][64];
  const int b = blockIdx.y;
  const int cap = p.max_blocks * p.page_size;
  const int len = clamped_len(p.seqlens, b, cap, blockIdx.x == 0 && threadIdx.x == 0);
  int n = p.new_lens ? p.new_lens[b] : min(p.Nn, len);
  if (n < 0 || n > p.Nn || n > len) {
    if (blockIdx.x == 0 && threadIdx.x == 0) record(2, kDevBadSeqlen);
    n = min(max(n, 0), min(p.Nn, len));
  }
  if (n == 0) return;
  const int blk = (len - n) / kBlock + static_cast<int>(blockIdx.x) / slabs;
  if (blk * kBlock >= len) return;
  const int pg = p.block_table[static_cast<long long>(b) * p.max_blocks + blk * kBlock / p.page_size];
  if (pg < 0 || pg >= p.num_pages) {
    if (threadIdx.x == 0) record(3, kDevBadPage);
    return;
  }
  const int row0 = blk * kBlock % p.page_size;
  const int rows = min(kBlock, len - blk * kBlock);
  const int per = p.Hkv * p.d / 8;  // chunks of a key row
  const int chunk = static_cast<int>(blockIdx.x) % slabs * 64 + (threadIdx.x & 63);
  const int g = threadIdx.x >> 6;
  const uint32_t inf2 = 0x7f807f80u, ninf2 = 0xff80ff80u;
  uint4 lo = make_uint4(inf2, inf2, inf2, inf2), hi = make_uint4(ninf2, ninf2, ninf2, ninf2);
  if (chunk < per) {
    const uint4* src = static_cast<const uint4*>(p.k_pages) +
                       (static_cast<long long>(pg) * p.page_size + row0 + 16 * g) * per + chunk;
    uint4 u[16];
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (16 * g + i < rows) u[i] = src[static_cast<long long>(i) * per];
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (16 * g + i < rows) {
        lo = min4(lo, u[i]);
        hi = max4(hi, u[i]);
      }
  }
  if (g > 0) {
    s_lo[g - 1][threadIdx.x & 63] = lo;
    s_hi[g - 1][threadIdx.x & 63] = hi;
  }
  __syncthreads();
  if (g == 0 && chunk < per) {
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      lo = min4(lo, s_lo[i][threadIdx.x]);
      hi = max4(hi, s_hi[i][threadIdx.x]);
    }
    const int dc = p.d / 8;
    uint4* dst = static_cast<uint4*>(p.k_bounds) +
                 ((static_cast<long long>(pg) * (p.page_size / kBlock) + row0 / kBlock) * p.Hkv + chunk / dc) * 2 * dc +
                 chunk % dc;
    dst[0] = lo;
    dst[dc] = hi;
  }
}

// ---------------------------------------------------------------------------
// Blocks of a query row.  A row is (token, KV head); token t = b * Nq + n.
struct RowSpan {
  int b, n, nb;  // sequence, new token, blocks that it sees (the last one its own)
};
__device__ __forceinline__ RowSpan row_span(const SelectParams& p, int token, bool report) {
  RowSpan r;
  r.b = token / p.Nq;
  r.n = token - r.b * p.Nq;
  const int len = clamped_len(p.seqlens, r.b, p.max_blocks * p.page_size, report);
  const int pos = len - p.Nq + r.n;
  r.nb = pos < 0 ? 0 : pos / kBlock + 1;
  return r;
}

// Bounds of block j of a sequence and KV head: lo [D], hi [D].
__device__ __forceinline__ const __nv_bfloat16* bounds_at(const SelectParams& p, int b, int j, int h) {
  const int per = p.page_size / kBlock;
  int pg = p.block_table[static_cast<long long>(b) * p.max_blocks + j / per];
  if (pg < 0 || pg >= p.num_pages) {
    record(4, kDevBadPage);
    pg = 0;
  }
  return static_cast<const __nv_bfloat16*>(p.k_bounds) +
         ((static_cast<long long>(pg) * per + j % per) * p.Hkv + h) * 2 * p.d;
}

// Scores on the tensor core.  For one sequence and KV head
//     S^T [128 blocks x N rows] = [lo hi] [q- q+]^T,
// 2 d deep, rows being tokens with the group's heads: a thread holds a block's
// scores (TMEM lane), so the largest over a token's heads is taken in its
// registers and a warp writes 32 neighbouring scores.  Many rows (N = 128): a CTA
// keeps its 128 blocks and walks the rows, bound by laying these out (2048 tokens
// of 32 heads, 512 blocks, 8 KV heads of d = 128: 40 us, 17 GFLOP).  Up to 64 rows
// (N = 16 or 64): a CTA keeps the rows and walks the blocks, the next ones on their
// way to registers while these are multiplied; bound by reading the bounds (16
// sequences of up to 128 K keys, 4 rows each: 75 MB in 24 us).  Measured on these
// sequences, us of the whole call, walking the blocks / the rows: 4 rows 37 / 84,
// 20 rows 57 / 100, 32 rows 67 / 104, 64 rows 98 / 127.
template <int D>
struct MmaLayout {
  static constexpr int N = 128;
  static constexpr int kA = 128 * 2 * D * 2, kB = N * 2 * D * 2;
  static constexpr int kBufs = 2;  // buffers of rows and of scores
  static constexpr int kThreads = 512;
  static constexpr int kOffB = kA;
  static constexpr int kOffNorm = kOffB + kBufs * kB;  // [kBufs][N] |q|^2, [128] |m|^2
  static constexpr int kOffBar = kOffNorm + (kBufs * N + 128) * 4;
  static constexpr int kOffPage = kOffBar + kBufs * 8 + 16;  // [128] where the blocks' bounds lie
  static constexpr int kBytes = kOffPage + 128 * 8;
  static constexpr int kAlloc = kBytes + 1024;
  static constexpr uint32_t kTmem = 512;  // a token's heads are read 8 at a time, past the last one
};
__device__ __forceinline__ float sum_squares(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  float s = bf16lo(a) * bf16lo(a);
  s = fmaf(bf16hi(a), bf16hi(a), s);
  s = fmaf(bf16lo(b), bf16lo(b), s);
  s = fmaf(bf16hi(b), bf16hi(b), s);
  s = fmaf(bf16lo(c), bf16lo(c), s);
  s = fmaf(bf16hi(c), bf16hi(c), s);
  s = fmaf(bf16lo(d), bf16lo(d), s);
  return fmaf(bf16hi(d), bf16hi(d), s);
}
__device__ __forceinline__ uint32_t max_abs_nan2(uint32_t a, uint32_t b) {
  return max_nan2(a & 0x7fff7fffu, b & 0x7fff7fffu);
}

template <int D>
__global__ void __launch_bounds__(MmaLayout<D>::kThreads, 1) score_mma_kernel(const SelectParams p, int token0, int tokens) {
  using L = MmaLayout<D>;
  constexpr int N = L::N;
  constexpr int kThreads = L::kThreads, kGroups = kThreads / 128;
  constexpr int kC = D / 8;  // 16-byte chunks of a row of D
  constexpr int kLoads = (N * kC + kThreads - 1) / kThreads;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  float* s_q = reinterpret_cast<float*>(smem + L::kOffNorm);
  float* s_m = s_q + L::kBufs * N;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kOffBar);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kOffBar + L::kBufs * 8);
  const __nv_bfloat16** s_at = reinterpret_cast<const __nv_bfloat16**>(smem + L::kOffPage);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int G = p.Hq / p.Hkv, h = blockIdx.y;
  grid_depends();
  // the launch's tokens of sequence b: n0 .. n1 - 1
  const int b = token0 / p.Nq + blockIdx.z;
  const int n0 = max(0, token0 - b * p.Nq), n1 = static_cast<int>(min(static_cast<long long>(p.Nq), token0 + static_cast<long long>(tokens) - static_cast<long long>(b) * p.Nq));
  const int tile_tokens = N / G, row_tiles = (n1 - n0 + tile_tokens - 1) / tile_tokens;
  const int block_tiles = (p.n_blocks + 127) / 128;
  const int part = blockIdx.x / block_tiles, parts = gridDim.x / block_tiles;
  const int j0 = (blockIdx.x - part * block_tiles) * 128;
  const int len = clamped_len(p.seqlens, b, p.max_blocks * p.page_size, blockIdx.x == 0 && h == 0 && tid == 0);
  auto blocks_seen = [&](int n) {  // by token n
    const int pos = len - p.Nq + n;
    return pos < 0 ? 0 : pos / kBlock + 1;
  };
  const int t0 = static_cast<int>(static_cast<long long>(row_tiles) * part / parts),
            t1 = static_cast<int>(static_cast<long long>(row_tiles) * (part + 1) / parts);
  if (t0 >= t1 || blocks_seen(min(n1, n0 + t1 * tile_tokens) - 1) <= j0) return;
  int first = t0;  // the first tile whose last token sees a block of these
  while (blocks_seen(min(n1, n0 + (first + 1) * tile_tokens) - 1) <= j0) ++first;
  if (tid == 0) {
    for (int i = 0; i < L::kBufs; ++i) mbar_init(bars + i, 1);
    mbar_fence_init();
  }
  if (warp == 0) {
    tmem_alloc(tmem_slot, L::kTmem);
    tmem_relinquish();
  }
  // the blocks' bounds: block r, chunk c of lo and of hi
  const int j_end = (len + kBlock - 1) / kBlock;
  if (tid < 128) s_at[tid] = j0 + tid < j_end ? bounds_at(p, b, j0 + tid, h) : nullptr;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 128 * kC / kThreads; ++i) {
    const int idx = i * kThreads + tid, r = idx / kC, c = idx % kC;
    uint4 lo = make_uint4(0u, 0u, 0u, 0u), hi = lo;
    const uint4* src = reinterpret_cast<const uint4*>(s_at[r]);
    if (src) {
      lo = src[c];
      hi = src[kC + c];
    }
    uint8_t* to = smem + (c >> 3) * (128 * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
    *reinterpret_cast<uint4*>(to) = lo;
    *reinterpret_cast<uint4*>(to + (D / 64) * (128 * 128)) = hi;
    float m = sum_squares(max_abs_nan2(lo.x, hi.x), max_abs_nan2(lo.y, hi.y), max_abs_nan2(lo.z, hi.z), max_abs_nan2(lo.w, hi.w));
#pragma unroll
    for (int o = kC / 2; o > 0; o >>= 1) m += __shfl_xor_sync(0xffffffffu, m, o);
    if (c == 0) s_m[r] = m;
  }
  uint4 held[kLoads];
  // this thread's chunks of a tile of rows: element offsets from the tile's first token, and their tokens
  int off[kLoads], tok_of[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int idx = i * kThreads + tid, r = idx / kC, c = idx % kC;
    tok_of[i] = r < tile_tokens * G ? r / G : 0x7fffffff;
    off[i] = r < tile_tokens * G ? (r / G * p.Hq + r % G) * kC + c : 0;
  }
  auto fetch = [&](int t) {
    const int n = n0 + t * tile_tokens, cnt = min(tile_tokens, n1 - n);
    const uint4* q = static_cast<const uint4*>(p.q) + ((static_cast<long long>(b) * p.Nq + n) * p.Hq + h * G) * kC;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) held[i] = tok_of[i] < cnt ? q[off[i]] : make_uint4(0u, 0u, 0u, 0u);
  };
  // whether this CTA finds the norms of a tile's rows: those that see the tile take turns
  auto norms = [&](int t) { return t % ((blocks_seen(min(n1, n0 + (t + 1) * tile_tokens) - 1) - 1) / 128 + 1) == j0 / 128; };
  auto stage = [&](int buf, bool norm) {
    uint8_t* base = smem + L::kOffB + buf * L::kB;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int idx = i * kThreads + tid, r = idx / kC, c = idx % kC;
      const uint4 u = held[i];
      if (norm) {
        float m = sum_squares(u.x, u.y, u.z, u.w);
#pragma unroll
        for (int o = kC / 2; o > 0; o >>= 1) m += __shfl_xor_sync(0xffffffffu, m, o);
        if (c == 0 && r < N) s_q[buf * N + r] = m;
      }
      if (r >= N) continue;
      uint8_t* to = base + (c >> 3) * (N * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
      *reinterpret_cast<uint4*>(to) = make_uint4(min_nan2(u.x, 0u), min_nan2(u.y, 0u), min_nan2(u.z, 0u), min_nan2(u.w, 0u));
      *reinterpret_cast<uint4*>(to + (D / 64) * (N * 128)) =
          make_uint4(max_nan2(u.x, 0u), max_nan2(u.y, 0u), max_nan2(u.z, 0u), max_nan2(u.w, 0u));
    }
  };
  fetch(first);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if (warp == 0) {  // every part of the rows finds the same
    float m_max = 0.f;
    for (int r = lane; r < 128; r += 32) m_max = fmaxf(m_max, s_m[r] == s_m[r] ? s_m[r] : INFINITY);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m_max = fmaxf(m_max, __shfl_xor_sync(0xffffffffu, m_max, o));
    if (lane == 0) p.m_norm[(static_cast<long long>(b) * p.Hkv + h) * block_tiles + j0 / 128] = m_max;
  }
  volatile int never = 0;
  for (int t = first, k = 0; t <= t1; ++t, ++k) {
    if (t < t1) {
      const int buf = k & 1;
      stage(buf, norms(t));
      fence_proxy_async_smem();
      tc_fence_before();
      __syncthreads();
      if (tid == 0) {
        tc_fence_after();
        const uint64_t a = sdesc_sw128(smem_u32(smem), 16, 1024), q = sdesc_sw128(smem_u32(smem + L::kOffB + buf * L::kB), 16, 1024);
#pragma unroll
        for (int kk = 0; kk < 2 * D / 16; ++kk)
          mma_bf16_ss(tmem + buf * N, a + (((kk >> 2) * (128 * 128) + (kk & 3) * 32) >> 4),
                      q + (((kk >> 2) * (N * 128) + (kk & 3) * 32) >> 4), idesc_bf16_f32(128, N, 0), kk > 0 ? 1u : 0u);
        mma_commit(bars + buf);
      }
      __syncwarp();
      if (t + 1 < t1) fetch(t + 1);
    }
    // results of the tile before
    if (k == 0) continue;
    const int d = t - 1, buf = (k - 1) & 1;
    if (!mbar_wait(bars + buf, ((k - 1) / 2) & 1, &never, kWaitLimitNs)) record(5, kDevTimeout);
    tc_fence_after();
    const int n = n0 + d * tile_tokens, cnt = min(tile_tokens, n1 - n);
    // each four warps take a part of the tokens
    const int c0 = cnt * (warp >> 2) / kGroups, c1 = cnt * ((warp >> 2) + 1) / kGroups;
    const uint32_t at = tmem + buf * N + (static_cast<uint32_t>(warp & 3) << 21);
    const int j = j0 + (warp & 3) * 32 + lane;
    const long long lrow0 = (static_cast<long long>(b) * p.Nq + n - token0) * p.Hkv + h;
    const int sees = j * kBlock - len + p.Nq - n;  // the first token of the tile that sees this block
    const long long pitch = static_cast<long long>(p.Hkv) * p.n_blocks;
    float* to = p.scores + (lrow0 + static_cast<long long>(c0) * p.Hkv) * p.n_blocks + j;
    auto put = [&](int c, float v) {
      if (c >= sees) *to = v;
      to += pitch;
    };
    // Up to four heads a group: 16 columns hold four tokens or more whole, so one load
    // gives their scores.  Larger groups: 8 columns a token at a time, for four tokens.
    // Measured, us of the whole call (2048 tokens, 512 blocks, 8 KV heads of d = 128),
    // by whole tokens / 8 columns a token: one head 78 / 88, two 86 / 95, three 95 / 106,
    // four 103 / 109, on 2048 blocks 445 / 470; eight 147 / 147.
    auto whole_groups = [&](auto g) {
      constexpr int kG = decltype(g)::value, kTok = 16 / kG;
      auto tokens_at = [&](int c, bool all) {
        uint32_t u[16];
        tmem_ld16(at + kG * c, u);
        tmem_wait_ld();
#pragma unroll
        for (int x = 0; x < kTok; ++x) {
          float best = __uint_as_float(u[kG * x]);
#pragma unroll
          for (int i = 1; i < kG; ++i) best = fmaxf(best, __uint_as_float(u[kG * x + i]));
          if (all || c + x < c1) put(c + x, best);
        }
      };
      int c = c0;
#pragma unroll 1
      for (; c + kTok <= c1; c += kTok) tokens_at(c, true);
      if (c < c1) tokens_at(c, false);
    };
    if (G == 1) {
      whole_groups(std::integral_constant<int, 1>());
    } else if (G == 2) {
      whole_groups(std::integral_constant<int, 2>());
    } else if (G == 3) {
      whole_groups(std::integral_constant<int, 3>());
    } else if (G == 4) {
      whole_groups(std::integral_constant<int, 4>());
    } else {
#pragma unroll 1
      for (int c = c0; c < c1; c += 4) {
        float best[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) best[x] = -INFINITY;
#pragma unroll 1
        for (int g = 0; g < G; g += 8) {
          uint32_t u[4][8];
#pragma unroll
          for (int x = 0; x < 4; ++x) tmem_ld8(at + min(c + x, c1 - 1) * G + g, u[x]);
          tmem_wait_ld();
#pragma unroll
          for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (g + i < G) best[x] = fmaxf(best[x], __uint_as_float(u[x][i]));
        }
#pragma unroll
        for (int x = 0; x < 4; ++x)
          if (c + x < c1) put(c + x, best[x]);
      }
    }
    if (tid < cnt && norms(d)) {
      float q = 0.f;
      for (int g = 0; g < G; ++g) {
        const float x = s_q[buf * N + tid * G + g];
        q = fmaxf(q, x == x ? x : INFINITY);
      }
      p.q_norm[lrow0 + static_cast<long long>(tid) * p.Hkv] = q;
    }
    tc_fence_before();
    __syncthreads();  // scores, rows and norms are read
  }
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, L::kTmem);
  }
}

template <int D, int kN>
struct FewLayout {
  static constexpr int N = kN;
  static constexpr int kA = 128 * 2 * D * 2, kB = N * 2 * D * 2;
  static constexpr int kOffB = kA;
  static constexpr int kOffNorm = kOffB + kB;             // [128] |m|^2, [N] |q|^2
  static constexpr int kOffPage = kOffNorm + (128 + N) * 4;  // [2][128] where the blocks' bounds lie
  static constexpr int kOffBar = kOffPage + 2 * 128 * 8;
  static constexpr int kBytes = kOffBar + 16;
  static constexpr int kAlloc = kBytes + 1024;
  static constexpr uint32_t kTmem = 2 * N;  // a token's heads are read 8 at a time, past the last one
};

// All rows of a sequence (at most N); block tiles part, part + parts, ...
template <int D, int kN>
__global__ void __launch_bounds__(kThreads, 2) score_few_kernel(const SelectParams p, int token0, int tokens) {
  using L = FewLayout<D, kN>;
  constexpr int N = L::N, kC = D / 8, kLoads = 128 * kC / kThreads;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  float* s_m = reinterpret_cast<float*>(smem + L::kOffNorm);
  float* s_q = s_m + 128;
  const uint4** s_at = reinterpret_cast<const uint4**>(smem + L::kOffPage);
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + L::kOffBar);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kOffBar + 8);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int G = p.Hq / p.Hkv, h = blockIdx.y;
  grid_depends();
  const int b = token0 / p.Nq + blockIdx.z;
  const int n0 = max(0, token0 - b * p.Nq), n1 = static_cast<int>(min(static_cast<long long>(p.Nq), token0 + static_cast<long long>(tokens) - static_cast<long long>(b) * p.Nq));
  const int cnt = n1 - n0;
  const int len = clamped_len(p.seqlens, b, p.max_blocks * p.page_size, blockIdx.x == 0 && h == 0 && tid == 0);
  const int pos = len - p.Nq + n1 - 1;                    // of the last token
  const int nb = pos < 0 ? 0 : pos / kBlock + 1;          // blocks that it sees
  const int tiles = (nb + 127) / 128, block_tiles = (p.n_blocks + 127) / 128;
  if (static_cast<int>(blockIdx.x) >= tiles) return;
  if (tid == 0) {
    mbar_init(bar, 1);
    mbar_fence_init();
  }
  if (warp == 0) {
    tmem_alloc(tmem_slot, L::kTmem);
    tmem_relinquish();
  }
  auto places = [&](int t, int buf) {  // threads 0 .. 127
    const int j = 128 * t + tid;
    s_at[buf * 128 + tid] = t < tiles && j < nb ? reinterpret_cast<const uint4*>(bounds_at(p, b, j, h)) : nullptr;
  };
  uint4 lo[kLoads], hi[kLoads];
  auto fetch = [&](int buf) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int idx = i * kThreads + tid;
      const uint4* src = s_at[buf * 128 + idx / kC];
      lo[i] = hi[i] = make_uint4(0u, 0u, 0u, 0u);
      if (src) {
        lo[i] = src[idx % kC];
        hi[i] = src[kC + idx % kC];
      }
    }
  };
  if (tid < 128) places(blockIdx.x, 0);
  // the rows: chunk c of row r
#pragma unroll 1
  for (int idx = tid; idx < N * kC; idx += kThreads) {
    const int r = idx / kC, c = idx % kC;
    uint4 u = make_uint4(0u, 0u, 0u, 0u);
    if (r < cnt * G)
      u = (static_cast<const uint4*>(p.q) + ((static_cast<long long>(b) * p.Nq + n0 + r / G) * p.Hq + h * G + r % G) * kC)[c];
    float m = sum_squares(u.x, u.y, u.z, u.w);
#pragma unroll
    for (int o = kC / 2; o > 0; o >>= 1) m += __shfl_xor_sync(0xffffffffu, m, o);
    if (c == 0) s_q[r] = m;
    uint8_t* to = smem + L::kOffB + (c >> 3) * (N * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
    *reinterpret_cast<uint4*>(to) = make_uint4(min_nan2(u.x, 0u), min_nan2(u.y, 0u), min_nan2(u.z, 0u), min_nan2(u.w, 0u));
    *reinterpret_cast<uint4*>(to + (D / 64) * (N * 128)) =
        make_uint4(max_nan2(u.x, 0u), max_nan2(u.y, 0u), max_nan2(u.z, 0u), max_nan2(u.w, 0u));
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const long long lrow0 = (static_cast<long long>(b) * p.Nq + n0 - token0) * p.Hkv + h;
  if (blockIdx.x == 0 && tid < cnt) {
    float q = 0.f;
    for (int g = 0; g < G; ++g) {
      const float x = s_q[tid * G + g];
      q = fmaxf(q, x == x ? x : INFINITY);
    }
    p.q_norm[lrow0 + static_cast<long long>(tid) * p.Hkv] = q;
  }
  fetch(0);
  volatile int never = 0;
#pragma unroll 1
  for (int t = blockIdx.x, k = 0; t < tiles; t += gridDim.x, ++k) {
    const int j0 = 128 * t;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int idx = i * kThreads + tid, r = idx / kC, c = idx % kC;
      uint8_t* to = smem + (c >> 3) * (128 * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
      *reinterpret_cast<uint4*>(to) = lo[i];
      *reinterpret_cast<uint4*>(to + (D / 64) * (128 * 128)) = hi[i];
      float m = sum_squares(max_abs_nan2(lo[i].x, hi[i].x), max_abs_nan2(lo[i].y, hi[i].y), max_abs_nan2(lo[i].z, hi[i].z),
                            max_abs_nan2(lo[i].w, hi[i].w));
#pragma unroll
      for (int o = kC / 2; o > 0; o >>= 1) m += __shfl_xor_sync(0xffffffffu, m, o);
      if (c == 0) s_m[r] = m;
    }
    if (tid < 128) places(t + gridDim.x, (k + 1) & 1);
    fence_proxy_async_smem();
    __syncthreads();
    if (tid == 0) {
      const uint64_t a = sdesc_sw128(smem_u32(smem), 16, 1024), q = sdesc_sw128(smem_u32(smem + L::kOffB), 16, 1024);
      tc_fence_after();
#pragma unroll
      for (int kk = 0; kk < 2 * D / 16; ++kk)
        mma_bf16_ss(tmem, a + (((kk >> 2) * (128 * 128) + (kk & 3) * 32) >> 4), q + (((kk >> 2) * (N * 128) + (kk & 3) * 32) >> 4),
                    idesc_bf16_f32(128, N, 0), kk > 0 ? 1u : 0u);
      mma_commit(bar);
    }
    __syncwarp();
    if (t + static_cast<int>(gridDim.x) < tiles) fetch((k + 1) & 1);
    if (warp == 7) {
      float m = 0.f;
#pragma unroll
      for (int r = 0; r < 4; ++r) m = fmaxf(m, s_m[32 * r + lane] == s_m[32 * r + lane] ? s_m[32 * r + lane] : INFINITY);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      if (lane == 0) p.m_norm[(static_cast<long long>(b) * p.Hkv + h) * block_tiles + t] = m;
    }
    if (!mbar_wait(bar, k & 1, &never, kWaitLimitNs)) record(5, kDevTimeout);
    tc_fence_after();
    // each four warps take a part of the tokens
    {
      const int j = j0 + (warp & 3) * 32 + lane;
      const uint32_t at = tmem + (static_cast<uint32_t>(warp & 3) << 21);
#pragma unroll 1
      for (int c = warp >> 2; c < cnt; c += 2) {
        float best = -INFINITY;
#pragma unroll 1
        for (int g = 0; g < G; g += 8) {
          uint32_t u[8];
          tmem_ld8(at + c * G + g, u);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (g + i < G) best = fmaxf(best, __uint_as_float(u[i]));
        }
        if (j * kBlock <= len - p.Nq + n0 + c) p.scores[(lrow0 + static_cast<long long>(c) * p.Hkv) * p.n_blocks + j] = best;
      }
    }
    tc_fence_before();
    __syncthreads();  // scores, bounds and norms are read
  }
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, L::kTmem);
  }
}

// ---------------------------------------------------------------------------
// Choice.
__device__ __forceinline__ uint32_t ordered(float x) {  // larger float, larger integer
  const uint32_t u = __float_as_uint(x);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t u) {
  return __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u);
}

// The 64-bit score of block j, formed by a warp; NaN ranks as +inf.
__device__ __forceinline__ double exact_score(const SelectParams& p, const RowSpan& r, int token, int h, int j) {
  const int lane = threadIdx.x & 31;
  const int G = p.Hq / p.Hkv;
  const __nv_bfloat16* kb = bounds_at(p, r.b, j, h);
  double best = -INFINITY;
  for (int g = 0; g < G; ++g) {
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q) + (static_cast<long long>(token) * p.Hq + h * G + g) * p.d;
    double s = 0.;
    for (int i = lane; i < p.d; i += 32) {
      const float x = __bfloat162float(q[i]);
      const double lo = __bfloat162float(kb[i]), hi = __bfloat162float(kb[p.d + i]);
      s += x != x ? static_cast<double>(x) : fmax(static_cast<double>(x), 0.) * hi + fmin(static_cast<double>(x), 0.) * lo;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (s != s) s = INFINITY;
    best = fmax(best, s);
  }
  return best;
}

// The same from sums of three fp32 numbers (products of bf16 are exact in fp32; an
// addition leaves its error in the second number, and that one's in the third:
// Knuth's two-sum, cascaded as in Ogita, Rump and Oishi's SumK with K = 3), where
// the row's scores lie well within fp32's range.  Off by (2 n 2^-24)^3 of the sum of
// magnitudes, 2^-48 for n = 128 terms, where double precision guarantees 2^-46; at
// many times its rate here.  (Two numbers lose 2^-43, and blocks that double
// precision tells apart came out in the wrong order.)
struct Triple {
  float h, m, l;
};
__device__ __forceinline__ float two_sum(float a, float b, float& err) {
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  err = __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t));
  return s;
}
__device__ __forceinline__ Triple add_to(Triple a, float x) {
  float e, f;
  const float h = two_sum(a.h, x, e), m = two_sum(a.m, e, f);
  return {h, m, __fadd_rn(a.l, f)};
}
// the same whichever comes first, so that all lanes of a sum end with the same
__device__ __forceinline__ Triple add_triples(Triple a, Triple b) {
  float e, f, g;
  const float h = two_sum(a.h, b.h, e), ab = two_sum(a.m, b.m, f), m = two_sum(ab, e, g);
  return {h, m, __fadd_rn(__fadd_rn(a.l, b.l), __fadd_rn(f, g))};
}
__device__ __forceinline__ double triple_score(const SelectParams& p, const RowSpan& r, int token, int h, int j) {
  // eight lanes a head, four heads at a time
  const int lane = threadIdx.x & 31, sub = lane & 7, chunks = p.d >> 6;
  const int G = p.Hq / p.Hkv;
  const uint4* kb = reinterpret_cast<const uint4*>(bounds_at(p, r.b, j, h));
  const uint4* qs = static_cast<const uint4*>(p.q) + (static_cast<long long>(token) * p.Hq + h * G) * (p.d >> 3);
  double best = -INFINITY;
#pragma unroll 1
  for (int g = lane >> 3; g < ((G + 3) & ~3); g += 4) {
    Triple s = {0.f, 0.f, 0.f};
#pragma unroll 1
    for (int c = 0; c < chunks; ++c) {
      const int at = c * 8 + sub;
      float x[8], lo[8], hi[8];
      unpack8(qs[(g < G ? g : 0) * (p.d >> 3) + at], x);
      unpack8(kb[at], lo);
      unpack8(kb[(p.d >> 3) + at], hi);
#pragma unroll
      for (int i = 0; i < 8; ++i) s = add_to(s, __fmul_rn(x[i], x[i] > 0.f ? hi[i] : lo[i]));
    }
#pragma unroll
    for (int o = 4; o > 0; o >>= 1)
      s = add_triples(s, {__shfl_xor_sync(0xffffffffu, s.h, o), __shfl_xor_sync(0xffffffffu, s.m, o),
                          __shfl_xor_sync(0xffffffffu, s.l, o)});
    best = fmax(best, static_cast<double>(s.h) + (static_cast<double>(s.m) + static_cast<double>(s.l)));  // (head 0 again past the last one)
  }
  best = fmax(best, __shfl_xor_sync(0xffffffffu, best, 8));
  return fmax(best, __shfl_xor_sync(0xffffffffu, best, 16));
}
// triples: whether the row's scores have fp32's range; a sum that is very small may
// all the same be one of products that fp32 does not hold.
__device__ __noinline__ double score_again(const SelectParams& p, const RowSpan& r, int token, int h, int j, bool triples) {
  if (triples) {
    const double s = triple_score(p, r, token, h, j);
    if (fabs(s) >= 0x1p-80) return s;
  }
  return exact_score(p, r, token, h, j);
}

// The largest |m|^2 of the blocks that a row sees, by a warp.
__device__ __forceinline__ float bounds_norm(const SelectParams& p, const RowSpan& r, int h) {
  const float* m = p.m_norm + (static_cast<long long>(r.b) * p.Hkv + h) * ((p.n_blocks + 127) / 128);
  float x = 0.f;
  for (int i = threadIdx.x & 31; i <= (r.nb - 1) / 128; i += 32) x = fmaxf(x, m[i]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}

// Twice the bound on the error of a row's scores: 2 * 2^-15 |q| |m|, a little for
// the roundings of the norms, and what 256 products below fp32's range lose.
// Infinite where norms are, and where they are not numbers; and where one's square
// lies below 2^-100, as then its terms may have passed below that range, while
// their products with the other side need not: above it 256 terms lost are 2^-18 of
// the square.
constexpr float kLeastSquare = 0x1p-100f;
__device__ __forceinline__ float band_of(float m_norm, float q_norm) {
  if (!(m_norm >= kLeastSquare && q_norm >= kLeastSquare)) return INFINITY;
  const float band = 6.2e-5f * sqrtf(m_norm) * sqrtf(q_norm) + 1e-35f;
  return band <= 3e38f ? band : INFINITY;
}

// Whether all heads of a row are zeros (a padded token): every score is then 0
// and the lowest indexes win, without 64-bit scores for all.  By a warp.
__device__ __forceinline__ bool zero_row(const SelectParams& p, int token, int h, int lrow) {
  if (p.q_norm[lrow] != 0.f) return false;
  const int chunks = p.Hq / p.Hkv * (p.d >> 3);
  const uint4* q = static_cast<const uint4*>(p.q) + (static_cast<long long>(token) * p.Hkv + h) * chunks;
  uint32_t any = 0;
  for (int i = threadIdx.x & 31; i < chunks; i += 32) any |= (q[i].x | q[i].y | q[i].z | q[i].w) & 0x7fff7fffu;
  return __any_sync(0xffffffffu, any != 0u) == 0;
}

constexpr int kHeld = 8192;   // scores kept in shared memory
constexpr int kBand = 1024;   // blocks scored again at most, else all by passes over 64-bit keys

__device__ __forceinline__ unsigned long long ordered64(double x) {
  const unsigned long long u = static_cast<unsigned long long>(__double_as_longlong(x + 0.));  // -0 as 0
  return u >> 63 ? ~u : u | (1ull << 63);
}

// A warp for a row of up to 32 K blocks, block 32 m + lane in element m of a lane.
// Bound by a warp's chain of instructions, each count of the keys waiting for the one
// before (512 blocks: 2.0 instructions an SM and cycle of 4), so by the warps there
// are: with 64 registers, eight CTAs an SM, 2048 tokens and 8 KV heads take 102 us on
// 512 blocks (115 with the 108 that the compiler takes by itself), 182 (235) on 1024,
// 445 (549) on 2048, although a thread then spills 0.3, 0.6, 0.9 and 3.4 KB for K = 8,
// 16, 32 and 64.
constexpr int kChooseWarps = 4;
template <int K>
__global__ void __launch_bounds__(32 * kChooseWarps, 8) choose_warp_kernel(const SelectParams p, int token0, int rows) {
  grid_depends();
  const int lane = threadIdx.x & 31;
  const int lrow = blockIdx.x * kChooseWarps + (threadIdx.x >> 5);
  if (lrow >= rows) return;
  const int h = lrow % p.Hkv, token = token0 + lrow / p.Hkv;
  const RowSpan r = row_span(p, token, false);
  int* out = p.blocks + (static_cast<long long>(token) * p.Hkv + h) * p.topk;
  if (r.nb <= p.topk) {
    for (int i = lane; i < p.topk; i += 32) out[i] = i < r.nb ? i : -1;
    return;
  }
  const int c0 = p.sink, c1 = r.nb - p.local, k = p.topk - p.sink - p.local;
  const float* scores = p.scores + static_cast<long long>(lrow) * p.n_blocks;
  uint32_t key[K];  // 0: no candidate
#pragma unroll
  for (int m = 0; m < K; ++m) {
    const int j = 32 * m + lane;
    key[m] = j >= c0 && j < c1 ? ordered(scores[j]) : 0u;
  }
  uint32_t in = 0, in2 = 0;  // chosen elements of this lane
  auto take = [&](int m) {
    if (m < 32)
      in |= 1u << m;
    else
      in2 |= 1u << (m - 32);
  };
  const float m_norm = k > 0 ? bounds_norm(p, r, h) : 0.f;
  if (k > 0 && m_norm < INFINITY && zero_row(p, token, h, lrow)) {
#pragma unroll
    for (int m = 0; m < K; ++m)
      if (32 * m + lane >= c0 && 32 * m + lane < c0 + k) take(m);
  } else if (k > 0) {
    const float band = band_of(m_norm, p.q_norm[lrow]);
    uint32_t lo = 1u, hi = 0xffffffffu;  // without a bound on the errors all candidates lie between
    if (band < 1e38f) {
      // the k-th largest, between t and t + 2^last - 1: the largest t with k keys
      // at or above it, from the bits that all keys share down to a quarter of the band
      uint32_t top = 0u, bottom = 0xffffffffu;
#pragma unroll
      for (int m = 0; m < K; ++m) {
        top = max(top, key[m]);
        bottom = min(bottom, key[m] ? key[m] : 0xffffffffu);
      }
      top = __reduce_max_sync(0xffffffffu, top);
      bottom = __reduce_min_sync(0xffffffffu, bottom);
      const float large = fmaxf(fabsf(unordered(top)), fabsf(unordered(bottom)));
      const int last = min(max(static_cast<int>(__float_as_uint(band) >> 23) - 2 - (static_cast<int>(__float_as_uint(large) >> 23) - 23), 0), 24);
      const int differ = 32 - __clz(top ^ bottom);  // bits from here on down
      uint32_t t = differ == 32 ? 0u : top >> differ << differ;
#pragma unroll 1
      for (int bit = differ - 1; bit >= last; --bit) {
        const uint32_t c = t | 1u << bit;
        int n = 0;
#pragma unroll
        for (int m = 0; m < K; ++m) n += key[m] >= c ? 1 : 0;
        if (__reduce_add_sync(0xffffffffu, n) >= k) t = c;
      }
      const uint32_t rest = differ > last ? (1u << last) - 1u : (differ == 32 ? 0xffffffffu : (1u << differ) - 1u);
      lo = max(ordered(unordered(t) - band), 1u);
      hi = ordered(unordered(t | rest) + band);
    }
    int sure = 0, between = 0;
#pragma unroll
    for (int m = 0; m < K; ++m) {
      sure += key[m] > hi ? 1 : 0;
      between += key[m] >= lo && key[m] <= hi ? 1 : 0;
    }
    sure = __reduce_add_sync(0xffffffffu, sure);
    between = __reduce_add_sync(0xffffffffu, between);
    const int left = k - sure;
#pragma unroll
    for (int m = 0; m < K; ++m)
      if (key[m] > hi || (between == left && key[m] >= lo)) take(m);
    if (between > left) {
      // those between, by their 64-bit scores (in sums of three fp32 where those have the range)
      const bool triples = band > 1e-18f && band < 1e18f;
      auto exact = [&](int j) { return ordered64(score_again(p, r, token, h, j, triples)); };
      if (between <= 32) {
        // a lane each
        unsigned long long u = 0;
        int n = 0, id = 0;
#pragma unroll
        for (int m = 0; m < K; ++m) {
          uint32_t w = __ballot_sync(0xffffffffu, key[m] >= lo && key[m] <= hi);
#pragma unroll 1
          while (w) {
            const int l = __ffs(w) - 1;
            w &= w - 1;
            const unsigned long long v = exact(32 * m + l);
            if (lane == n) {
              u = v;
              id = 32 * m + l;
            }
            ++n;
          }
        }
        int rank = 0;  // they are in the order of their indexes
#pragma unroll 1
        for (int o = 0; o < n; ++o) {
          const unsigned long long v = __shfl_sync(0xffffffffu, u, o);
          rank += v > u || (v == u && o < lane);
        }
        const uint32_t won = __ballot_sync(0xffffffffu, lane < n && rank < left);
#pragma unroll 1
        for (int o = 0; o < n; ++o) {
          const int j = __shfl_sync(0xffffffffu, id, o);
          if ((won >> o & 1u) && (j & 31) == lane) take(j >> 5);
        }
      } else {
        unsigned long long ex[K];  // 0: not between
#pragma unroll
        for (int m = 0; m < K; ++m) {
          ex[m] = 0;
          uint32_t w = __ballot_sync(0xffffffffu, key[m] >= lo && key[m] <= hi);
#pragma unroll 1
          while (w) {
            const int l = __ffs(w) - 1;
            w &= w - 1;
            const unsigned long long u = exact(32 * m + l);
            if (lane == l) ex[m] = u;
          }
        }
        unsigned long long t = 0;  // the largest that `left` of them reach
        int above = 0;             // those above it
#pragma unroll 1
        for (unsigned long long bit = 1ull << 63; bit; bit >>= 1) {
          int n = 0;
#pragma unroll
          for (int m = 0; m < K; ++m) n += ex[m] >= (t | bit) ? 1 : 0;
          if (__reduce_add_sync(0xffffffffu, n) >= left) t |= bit;
        }
#pragma unroll
        for (int m = 0; m < K; ++m) above += ex[m] > t ? 1 : 0;
        int equal = left - __reduce_add_sync(0xffffffffu, above);  // of those equal to it the first ones
#pragma unroll
        for (int m = 0; m < K; ++m) {
          const uint32_t same = __ballot_sync(0xffffffffu, ex[m] == t);
          if (ex[m] > t || (ex[m] == t && __popc(same & ((1u << lane) - 1u)) < equal)) take(m);
          equal -= min(equal, __popc(same));
        }
      }
    }
  }
  int at = 0;
#pragma unroll
  for (int m = 0; m < K; ++m) {
    const int j = 32 * m + lane;
    const bool c = j < r.nb && (j < c0 || j >= c1 || (m < 32 ? in >> m & 1u : in2 >> (m - 32) & 1u));
    const uint32_t w = __ballot_sync(0xffffffffu, c);
    if (c) out[at + __popc(w & ((1u << lane) - 1u))] = j;
    at += __popc(w);
  }
}
template <int K>
cudaError_t launch_choose_warp(const SelectParams& p, int token0, int rows, cudaStream_t stream) {
  return launch_dependent(choose_warp_kernel<K>, dim3(static_cast<unsigned>((rows + kChooseWarps - 1) / kChooseWarps)),
                          32 * kChooseWarps, 0, stream, p, token0, rows);
}

// One CTA for a row of more.  K > 0: up to 256 K candidates, whose keys stay in
// registers; 0: any number.
template <int K>
__global__ void __launch_bounds__(kThreads) choose_kernel(const SelectParams p, int token0) {
  grid_depends();
  extern __shared__ float s_score[];  // [min(n_blocks, kHeld)]
  __shared__ unsigned s_hist[256];
  __shared__ int s_pick, s_left, s_count[2];
  __shared__ uint32_t s_turn[2][kThreads / 32];
  __shared__ unsigned s_warp[kThreads / 32];
  __shared__ int s_id[kBand];
  __shared__ double s_exact[kBand];
  __shared__ uint32_t s_take[kBand / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int h = blockIdx.x % p.Hkv;
  const int token = token0 + static_cast<int>(blockIdx.x / p.Hkv);
  const int lrow = blockIdx.x;
  const RowSpan r = row_span(p, token, false);
  int* out = p.blocks + (static_cast<long long>(token) * p.Hkv + h) * p.topk;
  if (r.nb <= p.topk) {
    for (int i = tid; i < p.topk; i += kThreads) out[i] = i < r.nb ? i : -1;
    return;
  }
  // candidates [c0, c1), k of them wanted; sink + local <= topk < nb.  Those of a row of zeros are the first ones: k
  // more at the front, none of the others
  const float m_norm = bounds_norm(p, r, h);
  const bool zeros = m_norm < INFINITY && zero_row(p, token, h, lrow);
  const int all_k = p.topk - p.sink - p.local;
  const int c0 = p.sink + (zeros ? all_k : 0), c1 = r.nb - p.local, k = zeros ? 0 : all_k;
  const int n = c1 - c0;
  const float* scores = p.scores + static_cast<long long>(lrow) * p.n_blocks + c0;
  const bool held = n <= kHeld;
  if (held)
    for (int i = tid; i < n; i += kThreads) s_score[i] = scores[i];
  __syncthreads();
  auto score = [&](int i) { return held ? s_score[i] : scores[i]; };
  float t_lo = INFINITY, t_hi = INFINITY;  // chosen above t_hi, perhaps from t_lo on
  int mode = 0;                            // 0: nothing but scores > t_hi; 1: band scored again; 2: by passes
  unsigned long long cut = 0;              // mode 2: keys above it are in, of those equal the first `left`
  int left = 0;
  if (k > 0) {
    const float band = band_of(m_norm, p.q_norm[lrow]);
    const bool all = !(band < 1e38f), triples = band > 1e-18f && band < 1e18f;
    if (!all) {
      // the k-th largest, as in the warps' form: counts of the keys at or above a
      // value, a bit at a time
      uint32_t key[K > 0 ? K : 1];
      uint32_t top = 0u, bottom = 0xffffffffu;
      if constexpr (K > 0) {
#pragma unroll
        for (int m = 0; m < K; ++m) {
          const int i = m * kThreads + tid;
          key[m] = i < n ? ordered(s_score[i]) : 0u;
          top = max(top, key[m]);
          bottom = min(bottom, i < n ? key[m] : 0xffffffffu);
        }
      } else {
        for (int i = tid; i < n; i += kThreads) {
          const uint32_t u = ordered(score(i));
          top = max(top, u);
          bottom = min(bottom, u);
        }
      }
      top = __reduce_max_sync(0xffffffffu, top);
      bottom = __reduce_min_sync(0xffffffffu, bottom);
      if (lane == 0) {
        s_turn[0][warp] = top;
        s_turn[1][warp] = bottom;
      }
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kThreads / 32; ++w) {
        top = max(top, s_turn[0][w]);
        bottom = min(bottom, s_turn[1][w]);
      }
      __syncthreads();
      const float large = fmaxf(fabsf(unordered(top)), fabsf(unordered(bottom)));
      const int last = min(max(static_cast<int>(__float_as_uint(band) >> 23) - 2 - (static_cast<int>(__float_as_uint(large) >> 23) - 23), 0), 24);
      const int differ = 32 - __clz(top ^ bottom);  // bits from here on down
      uint32_t t0 = differ == 32 ? 0u : top >> differ << differ;
#pragma unroll 1
      for (int bit = differ - 1; bit >= last; --bit) {
        const uint32_t c = t0 | 1u << bit;
        int cnt = 0;
        if constexpr (K > 0) {
#pragma unroll
          for (int m = 0; m < K; ++m) cnt += key[m] >= c ? 1 : 0;
        } else {
          for (int i = tid; i < n; i += kThreads) cnt += ordered(score(i)) >= c ? 1 : 0;
        }
        cnt = __reduce_add_sync(0xffffffffu, cnt);
        if (lane == 0) s_turn[bit & 1][warp] = static_cast<uint32_t>(cnt);
        __syncthreads();
        cnt = 0;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) cnt += static_cast<int>(s_turn[bit & 1][w]);
        if (cnt >= k) t0 = c;
      }
      const uint32_t rest = differ > last ? (1u << last) - 1u : (differ == 32 ? 0xffffffffu : (1u << differ) - 1u);
      t_hi = unordered(t0 | rest) + band;
      t_lo = unordered(t0) - band;
    } else {
      t_hi = INFINITY;
      t_lo = -INFINITY;
    }
    // how many are in for sure, and the blocks between
    if (tid < 2) s_count[tid] = 0;
    if (tid < kBand / 32) s_take[tid] = 0;
    __syncthreads();
    int sure = 0;
    for (int i = tid; i < n; i += kThreads) {
      const float x = score(i);
      if (!all && x > t_hi) {
        ++sure;
      } else if (all || x >= t_lo) {
        const int at = atomicAdd(&s_count[1], 1);
        if (at < kBand) s_id[at] = i;
      }
    }
    if (sure) atomicAdd(&s_count[0], sure);
    __syncthreads();
    const int between = s_count[1];
    left = k - s_count[0];
    if (between > left) {
      if (between <= kBand) {
        mode = 1;
        for (int m = warp; m < between; m += kThreads / 32) {
          const double x = score_again(p, r, token, h, c0 + s_id[m], triples);
          if (lane == 0) s_exact[m] = x;
        }
        __syncthreads();
        for (int m = tid; m < between; m += kThreads) {
          const double x = s_exact[m];
          const int id = s_id[m];
          int rank = 0;
          for (int o = 0; o < between; ++o) rank += s_exact[o] > x || (s_exact[o] == x && s_id[o] < id);
          if (rank < left) atomicOr(&s_take[m >> 5], 1u << (m & 31));
        }
        __syncthreads();
        // the taken ones get a score above all: marked in place of their number
        for (int m = tid; m < between; m += kThreads)
          if (!(s_take[m >> 5] >> (m & 31) & 1u)) s_id[m] = -1;
      } else {
        mode = 2;
        int want = left;
        for (int shift = 56; shift >= 0; shift -= 8) {
          s_hist[tid] = 0;
          __syncthreads();
          for (int i = warp; i < n; i += kThreads / 32) {
            const float x = score(i);
            if (!all && !(x >= t_lo && x <= t_hi)) continue;
            const unsigned long long u = ordered64(score_again(p, r, token, h, c0 + i, false));
            if (lane == 0 && (shift == 56 || (u >> (shift + 8)) == cut)) atomicAdd(&s_hist[(u >> shift) & 255u], 1u);
          }
          __syncthreads();
          if (tid == 0) {
            int c = want;
            int v = 255;
            while (static_cast<int>(s_hist[v]) < c) c -= static_cast<int>(s_hist[v--]);
            s_pick = v;
            s_left = c;
          }
          __syncthreads();
          cut = (cut << 8) | static_cast<unsigned>(s_pick);
          want = s_left;
          __syncthreads();
        }
        left = want;
      }
    } else {
      t_hi = -INFINITY;  // everything from t_lo on
    }
  }
  // the chosen blocks in ascending order
  if (mode != 2 && r.nb <= kHeld) {
    // a bit for each, the words' sums, then each to its place
    __shared__ uint32_t s_bits[kHeld / 32];
    __shared__ int s_before[kHeld / 32];
    const int words = (r.nb + 31) >> 5;
    for (int base = 0; base < r.nb; base += kThreads) {
      const int j = base + tid, i = j - c0;
      bool in = j < r.nb && (j < c0 || j >= c1);
      if (k > 0 && i >= 0 && i < n) in = mode == 0 ? score(i) >= t_lo : score(i) > t_hi;
      const unsigned vote = __ballot_sync(0xffffffffu, in);
      if (lane == 0) s_bits[(base >> 5) + warp] = vote;
    }
    __syncthreads();
    if (mode == 1)
      for (int m = tid; m < s_count[1]; m += kThreads)
        if (s_id[m] >= 0) atomicOr(&s_bits[(s_id[m] + c0) >> 5], 1u << ((s_id[m] + c0) & 31));
    __syncthreads();
    if (warp == 0) {
      int sum = 0;
      for (int w0 = 0; w0 < words; w0 += 32) {
        const int mine = w0 + lane < words ? __popc(s_bits[w0 + lane]) : 0;
        int incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int x = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += x;
        }
        if (w0 + lane < words) s_before[w0 + lane] = sum + incl - mine;
        sum += __shfl_sync(0xffffffffu, incl, 31);
      }
    }
    __syncthreads();
    for (int j = tid; j < r.nb; j += kThreads) {
      const uint32_t w = s_bits[j >> 5];
      if (w >> lane & 1u) out[s_before[j >> 5] + __popc(w & ((1u << lane) - 1u))] = j;
    }
    return;
  }
  __shared__ int s_done, s_equal;
  if (tid == 0) s_done = s_equal = 0;
  __syncthreads();
  for (int base = 0; base < r.nb; base += kThreads) {
    const int j = base + tid, i = j - c0;
    bool in = j < r.nb && (j < c0 || j >= c1);
    if (k > 0 && i >= 0 && i < n) {
      const float x = score(i);
      if (mode == 0)
        in = x >= t_lo;
      else
        in = x > t_hi;
    }
    if (mode == 1) {
      // numbers of this stretch among the taken ones
      __shared__ uint32_t s_bits[kThreads / 32];
      if (tid < kThreads / 32) s_bits[tid] = 0;
      __syncthreads();
      for (int m = tid; m < s_count[1]; m += kThreads) {
        const int at = s_id[m] < 0 ? -1 : s_id[m] + c0 - base;
        if (at >= 0 && at < kThreads) atomicOr(&s_bits[at >> 5], 1u << (at & 31));
      }
      __syncthreads();
      in = in || (s_bits[warp] >> lane & 1u);
      __syncthreads();
    } else if (mode == 2) {
      // each warp scores its 32 blocks again; equal ones are counted in order
      uint32_t above = 0, equal = 0;
      for (int o = 0; o < 32; ++o) {
        const int io = base + warp * 32 + o - c0;
        if (io < 0 || io >= n) continue;
        const float x = score(io);
        const bool certain = t_hi < INFINITY && x > t_hi;
        if (certain || (t_lo > -INFINITY && x < t_lo)) continue;
        const unsigned long long u = ordered64(score_again(p, r, token, h, c0 + io, false));
        if (u > cut) above |= 1u << o;
        if (u == cut) equal |= 1u << o;
      }
      if (lane == 0) s_warp[warp] = equal;
      __syncthreads();
      int before = s_equal;
      for (int w = 0; w < warp; ++w) before += __popc(s_warp[w]);
      before += __popc(equal & ((1u << lane) - 1u));
      in = in || (above >> lane & 1u) || ((equal >> lane & 1u) && before < left);
      __syncthreads();
      if (tid == 0)
        for (int w = 0; w < kThreads / 32; ++w) s_equal += __popc(s_warp[w]);
      __syncthreads();
    }
    const unsigned vote = __ballot_sync(0xffffffffu, in);
    if (lane == 0) s_warp[warp] = vote;
    __syncthreads();
    int at = s_done;
    for (int w = 0; w < warp; ++w) at += __popc(s_warp[w]);
    at += __popc(vote & ((1u << lane) - 1u));
    if (in && at < p.topk) out[at] = j;
    __syncthreads();
    if (tid == 0)
      for (int w = 0; w < kThreads / 32; ++w) s_done += __popc(s_warp[w]);
    __syncthreads();
  }
}

}  // namespace

cudaError_t launch_key_bounds(const KeyBoundsParams& p, cudaStream_t stream) {
  const int slabs = (p.Hkv * p.d / 8 + 63) / 64;
  const long long cap = static_cast<long long>(p.max_blocks) * p.page_size;
  const long long most = p.Nn < cap ? p.Nn : cap;
  const long long blocks = (most + kBlock - 2) / kBlock + 1;
  return launch_dependent(bounds_kernel, dim3(static_cast<unsigned>(blocks * slabs), static_cast<unsigned>(p.B)), kThreads,
                          0, stream, p, slabs);
}

template <int D, int N>
cudaError_t launch_score_few(const SelectParams& p, int token0, int tokens, cudaStream_t stream) {
  using L = FewLayout<D, N>;
  auto kern = score_few_kernel<D, N>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kAlloc);
  if (e != cudaSuccess) return e;
  const int seqs = (token0 + tokens - 1) / p.Nq - token0 / p.Nq + 1, block_tiles = (p.n_blocks + 127) / 128;
  // two CTAs an SM, twice: sequences differ in their blocks
  const long long others = static_cast<long long>(p.Hkv) * seqs;
  long long parts = others >= 608 ? 1 : (608 + others - 1) / others;
  if (parts > block_tiles) parts = block_tiles;
  return launch_dependent(kern, dim3(static_cast<unsigned>(parts), static_cast<unsigned>(p.Hkv), static_cast<unsigned>(seqs)),
                          kThreads, L::kAlloc, stream, p, token0, tokens);
}

template <int D>
cudaError_t launch_score_mma(const SelectParams& p, int token0, int tokens, cudaStream_t stream) {
  using L = MmaLayout<D>;
  constexpr int N = L::N;
  auto kern = score_mma_kernel<D>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kAlloc);
  if (e != cudaSuccess) return e;
  const int seqs = (token0 + tokens - 1) / p.Nq - token0 / p.Nq + 1;
  const int block_tiles = (p.n_blocks + 127) / 128, tile_tokens = N / (p.Hq / p.Hkv);
  const long long row_tiles = ((tokens < p.Nq ? tokens : p.Nq) + tile_tokens - 1) / tile_tokens;
  // the rows in as many parts as fill the SMs once, not twice
  const long long others = static_cast<long long>(block_tiles) * p.Hkv * seqs;
  long long parts = others >= 152 ? 1 : 152 / others;
  if (parts > row_tiles) parts = row_tiles;
  return launch_dependent(kern, dim3(static_cast<unsigned>(block_tiles * parts), static_cast<unsigned>(p.Hkv), static_cast<unsigned>(seqs)),
                          L::kThreads, L::kAlloc, stream, p, token0, tokens);
}

cudaError_t launch_select(const SelectParams& p, int token0, int tokens, cudaStream_t stream) {
  const int rows = p.Nq * (p.Hq / p.Hkv);
  cudaError_t e;
  if (rows <= 16)
    e = p.d == 64 ? launch_score_few<64, 16>(p, token0, tokens, stream) : launch_score_few<128, 16>(p, token0, tokens, stream);
  else if (rows <= 64)
    e = p.d == 64 ? launch_score_few<64, 64>(p, token0, tokens, stream) : launch_score_few<128, 64>(p, token0, tokens, stream);
  else
    e = p.d == 64 ? launch_score_mma<64>(p, token0, tokens, stream) : launch_score_mma<128>(p, token0, tokens, stream);
  if (e != cudaSuccess) return e;
  const int n = tokens * p.Hkv;
  // More rows than blocks: a warp a row; fewer: a CTA a row.  Measured, us of the whole call, a warp / a CTA:
  //     512 blocks: 128 rows 27.8 / 24.3, 256 21.3 / 18.9, 512 21.6 / 25.0, 1024 24.2 / 34.4, 16384 103 / 362
  //     1024: 128 rows 41.9 / 33.8;  2048: 128 rows 50.2 / 36.9, 2048 127 / 126, 16384 446 / 589
  // (128 rows: 16 sequences, the others one).
  if (n > p.n_blocks) {
    if (p.n_blocks <= 256) return launch_choose_warp<8>(p, token0, n, stream);
    if (p.n_blocks <= 512) return launch_choose_warp<16>(p, token0, n, stream);
    if (p.n_blocks <= 1024) return launch_choose_warp<32>(p, token0, n, stream);
    if (p.n_blocks <= 2048) return launch_choose_warp<64>(p, token0, n, stream);
  }
  const int held = p.n_blocks < kHeld ? p.n_blocks : kHeld;
  return launch_dependent(p.n_blocks <= 8 * kThreads ? choose_kernel<8> : choose_kernel<0>, dim3(static_cast<unsigned>(n)), kThreads,
                          held * static_cast<int>(sizeof(float)), stream, p, token0);
}

cudaError_t status_word_select(uint32_t** at) { return cudaGetSymbolAddress(reinterpret_cast<void**>(at), g_select_status); }

}  // namespace attn

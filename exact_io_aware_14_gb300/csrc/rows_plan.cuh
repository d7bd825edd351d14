// What the kernels of attention over a paged bf16 cache share: their work, cut
// into equal runs of key tiles, and their waits.  Included by each of those
// units, each with a status word of its own.
#pragma once
#include <cuda_runtime.h>

#include "launch.h"
#include "ptx.cuh"

namespace attn {
namespace {

__device__ uint32_t g_rows_status;

__device__ __forceinline__ void record(uint32_t site, uint32_t code) {
  atomicCAS(&g_rows_status, 0u, (site << 8) | code);
}

constexpr uint64_t kWaitLimitNs = 2000000000ull;  // 2 s: no legitimate wait comes close
constexpr int kMaskWords = kMaxListed / 32;

// Value rows to clear: behind the keys that count they hold anything, NaN
// included, and P = 0 times NaN is not 0; halves that were not loaded hold older
// tiles.
struct Fix {
  int slot, v0, v1;  // ring slot (-1: no more); value rows that count of its two halves
};
// Start of a CTA's lanes, set up by all threads.
struct Plan {
  long long lane_at[2];  // tiles from the start of the sequence's keys
  int lane_b[2];         // sequence at which the lanes start (-1: the prefix)
  long long total, pair_total;
  int prefix_end;        // keys of the prefix that any sequence has
  int all_see;           // keys that every row sees
};

// Bounded waits: one probe in line, the rest out of line, as the warps' code
// together has to fit the instruction cache (with 57% of its fetches hitting it
// a CTA's tile took three times as long).
__device__ __noinline__ bool wait_long(uint64_t* bar, uint32_t parity, volatile int* abort_flag, uint32_t site) {
  const bool ok = mbar_wait(bar, parity, abort_flag, kWaitLimitNs);
  if (!ok) record(site, kDevTimeout);
  return ok;
}
__device__ __forceinline__ bool wait_one(uint64_t* bar, uint32_t parity, volatile int* abort_flag, uint32_t site) {
  return mbar_test_wait(bar, parity) || wait_long(bar, parity, abort_flag, site);
}
__device__ __forceinline__ bool wait_all(uint64_t* bar, uint32_t parity, volatile int* abort_flag, uint32_t site) {
  return __all_sync(0xffffffffu, wait_one(bar, parity, abort_flag, site));
}

__device__ __forceinline__ int clamped_len(const RowsParams& p, int b) {
  return min(max(p.seqlens[b], 0), p.max_blocks * p.page_size);
}
__device__ __forceinline__ int tiles_of(int keys) { return (keys + 127) >> 7; }
// Key tiles of a sequence behind the prefix.
__device__ __forceinline__ int own_tiles(const RowsParams& p, int b) {
  return tiles_of(max(0, clamped_len(p, b) - p.shared_len));
}
// `total` tiles dealt to `lanes` in runs of equal length, none of them empty but
// the last ones: where run i starts, and which run holds tile x.
__device__ __noinline__ long long quotient(long long a, long long b) {  // a >= 0, b > 0; 64-bit divisions only where needed
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}
__device__ __forceinline__ long long run_start(long long total, int lanes, int i) {
  const long long runs = min(total, static_cast<long long>(lanes));
  return i < runs ? quotient(total * i, runs) : total;
}
__device__ __forceinline__ int run_of(long long total, int lanes, long long x) {
  const long long runs = min(total, static_cast<long long>(lanes));
  return static_cast<int>(quotient((x + 1) * runs - 1, total));
}

// Lanes' starts for ranges: sums of the sequences' tiles, by all threads of the
// CTA (kWarps warps, kSlots lanes a CTA: lane slot * grid + CTA).  CTA 0 leaves
// the sums before each sequence, and the totals, for the joining kernel.
template <int kWarps, int kSlots>
__device__ void make_plan(const RowsParams& p, Plan* plan, long long* s_sum, int* s_max) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kThreads = 32 * kWarps;
  const int per = p.Hkv * p.own_rt;  // units of a sequence
  // sums and extremes of all sequences; those of up to kThreads are scanned on the way
  const bool once = p.B <= kThreads;
  long long sum = 0, first = 0;
  int longest = 0, shortest = 0x7fffffff;
#pragma unroll 1
  for (int b = tid; b < p.B; b += kThreads) {
    const int raw = p.seqlens[b], len = min(max(raw, 0), p.max_blocks * p.page_size);
    first = static_cast<long long>(tiles_of(max(0, len - p.shared_len))) * per;
    sum += first;
    longest = max(longest, len);
    shortest = min(shortest, len);
    if (blockIdx.x == 0 && raw != len) record(1, kDevBadSeqlen);
  }
  longest = __reduce_max_sync(0xffffffffu, longest);
  shortest = __reduce_min_sync(0xffffffffu, shortest);
  // inclusive over the lanes of the warp: its last lane holds the warp's sum
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += y;
  }
  if (lane == 31) {
    s_sum[warp] = sum;
    s_max[warp] = longest;
    s_max[kWarps + warp] = shortest;
  }
  __syncthreads();
  long long all = 0, ahead = 0;
#pragma unroll 1
  for (int w = 0; w < kWarps; ++w) {
    if (w == warp) ahead = all;
    all += s_sum[w];
    longest = max(longest, s_max[w]);
    shortest = min(shortest, s_max[kWarps + w]);
  }
  const int end = min(p.shared_len, longest);
  const long long prefix = static_cast<long long>(tiles_of(end)) * p.Hkv;
  const long long solo = p.pairs ? 0 : prefix;
  const long long total = solo + all;
  if (tid == 0) {
    plan->prefix_end = end;
    plan->all_see = max(0, shortest - p.Nq + 1);
    plan->total = total;
    plan->pair_total = p.pairs ? prefix * p.pairs : 0;
  }
  if (blockIdx.x == 0 && tid == 0) {
    p.sums[p.B] = total;
    p.sums[p.B + 1] = p.pairs ? prefix * p.pairs : 0;
    p.sums[p.B + 2] = end;
  }
  long long x[kSlots];
  for (int s = 0; s < kSlots; ++s) {
    x[s] = run_start(total, kSlots * gridDim.x, s * gridDim.x + blockIdx.x);
    if (tid == 0 && x[s] < solo) {
      plan->lane_b[s] = -1;
      plan->lane_at[s] = x[s];
    }
  }
  auto place = [&](int b, long long before, long long mine) {
    if (blockIdx.x == 0) p.sums[b] = before;
    for (int s = 0; s < kSlots; ++s)
      if (before <= x[s] && x[s] < before + mine) {
        plan->lane_b[s] = b;
        plan->lane_at[s] = x[s] - before;
      }
  };
  if (once) {
    if (tid < p.B) place(tid, solo + ahead + sum - first, first);
    return;
  }
  long long base = solo;
#pragma unroll 1
  for (int b0 = 0; b0 < p.B; b0 += kThreads) {
    // the last slot's lane starts last; CTA 0 needs all sums
    if (blockIdx.x != 0 && base > x[kSlots - 1]) break;
    const int b = b0 + tid;
    const long long mine = b < p.B ? static_cast<long long>(own_tiles(p, b)) * per : 0;
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    __syncthreads();
    if (lane == 31) s_sum[warp] = incl;
    __syncthreads();
    long long before = base + incl - mine, chunk = 0;
#pragma unroll 1
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += s_sum[w];
      chunk += s_sum[w];
    }
    if (b < p.B) place(b, before, mine);
    base += chunk;
  }
}

// A place in the ring: slot and number of the turn through it.
template <int NS>
struct RingAt {
  uint32_t slot = 0, turn = 0;
  __device__ __forceinline__ void next() {
    if (++slot == NS) {
      slot = 0;
      ++turn;
    }
  }
};

// A K or V tile to load.
struct Tile {
  int g0, g1;      // first groups of 8 keys in the pool
  uint32_t flags;  // bits 0, 1: seen; 2, 3: seen whole
  int part;        // keys seen of those seen in part
};

// Block `blk` of table row `row`, as its first group of 8 keys in the pool.
__device__ __forceinline__ int pool_group(const RowsParams& p, int row, int blk) {
  const int at_page = blk * 64 / p.page_size;
  int g = p.block_table[static_cast<long long>(row) * p.max_blocks + at_page];
  if (g < 0 || g >= p.num_pages) {
    record(2, kDevBadPage);
    g = 0;
  }
  return g * (p.page_size / 8) + 8 * (blk - at_page * (p.page_size / 64));
}

}  // namespace
}  // namespace attn

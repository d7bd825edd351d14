// Attention of query rows over a paged bf16 cache, for sm_103a: over whole
// sequences whose first keys the batch shares (attn_fwd_splitkv_paged_shared),
// or over listed 64-key blocks (attn_fwd_blocks_paged).
//
// A row is a query token and one of the heads that read a KV head.  S = Q K^T
// and O += P V run on tcgen05 with 128 rows and 128 keys a tile.  The rows of a
// tile are all that read the same keys: for the shared prefix the tokens of the
// whole batch with the heads of a group, for a sequence's own keys its new
// tokens with theirs, for listed blocks one token's heads.  Where those are few
// most of a tile's rows are empty; their products cost what a full tile's do,
// 1024 cycles for 128 keys of d = 128, less than the 64 KB of K and V take to
// arrive (1.4 us at this SM's share of memory).
//
// Work is cut into equal runs of tiles, whatever the lengths.  A CTA has two
// slots, each with a tile of rows, its scores, its accumulator and a
// warpgroup for its softmax.
//   Pair work (a prefix read by more rows than one tile): the slots hold two
//     tiles of rows and share every K/V tile; each CTA takes an equal run of
//     (KV head, pair, key tile).
//   Lane work (all else): each slot is a lane of its own with its own K/V
//     tiles, and each lane takes an equal run of (unit, key tile), a unit being
//     the rows and keys named above.
// What a lane computes of a unit is a piece; pieces of a row (normalised O and
// log-sum-exp, fp32) go to the workspace, and a second kernel joins them in
// order.  A piece of listed blocks that is a whole unit is written as result.
// Piece numbers need no counters: along the runs either the lane or the unit
// goes up by one, so lane + unit is a number of its own for each piece.
//
// Warps: 0 producer (work, pages, TMA loads into one ring in the order of use),
// 1 MMA issuer, 2 clears value rows that hold anything, 4-7 and 8-11 softmax
// and results of slots 0 and 1.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "launch.h"
#include "ptx.cuh"
#include "rows_softmax.cuh"

namespace attn {
namespace {

__device__ uint32_t g_rows_status;

__device__ __forceinline__ void record(uint32_t site, uint32_t code) {
  atomicCAS(&g_rows_status, 0u, (site << 8) | code);
}

constexpr int kThreads = 384;
constexpr uint64_t kWaitLimitNs = 2000000000ull;  // 2 s: no legitimate wait comes close
constexpr uint32_t kTmemCols = 512;
constexpr int kMaskWords = kMaxListed / 32;

// What a slot computes next, as the producer tells the other warps.
struct Piece {
  int n;      // key tiles; -1: no more work
  int share;  // 0 own K/V tiles; 1 those of both slots; 2 the same, slot 1 without rows
  int h;      // KV head
  int tok0, ntok;  // first token, tokens
  int key0, keys;  // ranges: position of the first tile's first key, keys from there on
  int dst;    // piece number, -1: the result itself
  int part;   // keys seen of the blocks marked in part[] (lists)
  uint32_t full[kMaskWords], some[kMaskWords];  // lists: blocks seen whole, seen in part
};
struct Fix {
  int slot, v0, v1;  // ring slot; value rows that count of its two halves
};
// Start of the slots' lanes, set up by all threads.
struct Plan {
  long long lane_at[2];  // tiles from the start of the sequence's keys
  int lane_b[2];         // sequence at which the lanes start (-1: the prefix)
  long long total, pair_total;
  int prefix_end;        // keys of the prefix that any sequence has
};

template <int D>
struct Layout {
  static constexpr int kSlots = D == 64 ? 10 : 5;
  static constexpr int kHalf = 128 * 128;  // one 64-column block of a 128-row tile
  static constexpr int kTile = 128 * D * 2;
  static constexpr int kOffRing = 2 * kTile;
  static constexpr int kOffPiece = kOffRing + kSlots * kTile;
  static constexpr int kOffBar = kOffPiece + 4 * static_cast<int>(sizeof(Piece));
  static constexpr int kNumBars = 2 * kSlots + 4 * 2 + 4 * 4 + 3 * 4 + 1;
  static constexpr int kOffFix = kOffBar + 8 * kNumBars;
  static constexpr int kOffPlan = (kOffFix + 4 * static_cast<int>(sizeof(Fix)) + 15) & ~15;
  static constexpr int kOffScan = kOffPlan + static_cast<int>(sizeof(Plan));
  static constexpr int kOffMisc = kOffScan + 12 * 8 + 12 * 4;
  static constexpr int kBytes = kOffMisc + 16;
  static constexpr int kAlloc = kBytes + 1024;  // slack to align the base to 1024 B
};
static_assert(Layout<128>::kAlloc <= 232448 && Layout<64>::kAlloc <= 232448, "shared memory of a CTA");

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
__device__ __forceinline__ long long run_start(long long total, int lanes, int i) {
  const long long runs = min(total, static_cast<long long>(lanes));
  return i < runs ? total * i / runs : total;
}
__device__ __forceinline__ int run_of(long long total, int lanes, long long x) {
  const long long runs = min(total, static_cast<long long>(lanes));
  return static_cast<int>(((x + 1) * runs - 1) / total);
}
// The lane of a slot: with few runs the CTAs have one each.
__device__ __forceinline__ int lane_of(int slot) { return slot * static_cast<int>(gridDim.x) + static_cast<int>(blockIdx.x); }

// Lanes' starts for ranges: sums of the sequences' tiles, by all threads.  CTA 0
// leaves the sums before each sequence, and the totals, for the second kernel.
__device__ void make_plan(const RowsParams& p, Plan* plan, long long* s_sum, int* s_max) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kWarps = kThreads / 32;
  const int per = p.Hkv * p.own_rt;  // units of a sequence
  long long sum = 0;
  int longest = 0;
  for (int b = tid; b < p.B; b += kThreads) {
    sum += static_cast<long long>(own_tiles(p, b)) * per;
    longest = max(longest, clamped_len(p, b));
    if (blockIdx.x == 0 && (p.seqlens[b] < 0 || p.seqlens[b] > p.max_blocks * p.page_size)) record(1, kDevBadSeqlen);
  }
  longest = __reduce_max_sync(0xffffffffu, longest);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) {
    s_sum[warp] = sum;
    s_max[warp] = longest;
  }
  __syncthreads();
  sum = 0;
  for (int w = 0; w < kWarps; ++w) {
    sum += s_sum[w];
    longest = max(longest, s_max[w]);
  }
  const int end = min(p.shared_len, longest);
  const long long prefix = static_cast<long long>(tiles_of(end)) * p.Hkv;
  const long long solo = p.pairs ? 0 : prefix;
  const long long total = solo + sum;
  const int lanes = 2 * gridDim.x;
  if (tid == 0) {
    plan->prefix_end = end;
    plan->total = total;
    plan->pair_total = p.pairs ? prefix * p.pairs : 0;
  }
  if (blockIdx.x == 0 && tid == 0) {
    p.sums[p.B] = total;
    p.sums[p.B + 1] = p.pairs ? prefix * p.pairs : 0;
    p.sums[p.B + 2] = end;
  }
  long long x[2];
  for (int s = 0; s < 2; ++s) {
    x[s] = run_start(total, lanes, lane_of(s));
    if (tid == 0 && x[s] < solo) {
      plan->lane_b[s] = -1;
      plan->lane_at[s] = x[s];
    }
  }
  long long base = solo;
  for (int b0 = 0; b0 < p.B; b0 += kThreads) {
    // slot 1's lane starts last; CTA 0 needs all sums
    if (blockIdx.x != 0 && base > x[1]) break;
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
    long long before = base + incl - mine, all = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += s_sum[w];
      all += s_sum[w];
    }
    if (b < p.B && blockIdx.x == 0) p.sums[b] = before;
    for (int s = 0; s < 2; ++s)
      if (b < p.B && before <= x[s] && x[s] < before + mine) {
        plan->lane_b[s] = b;
        plan->lane_at[s] = x[s] - before;
      }
    base += all;
  }
}

// Where a lane stands in its run (all lanes of the producer warp alike).
struct Lane {
  long long left;       // ranges: tiles left
  long long unit, end;  // lists: next whole unit and their end; then the cut ones
  int b, h, rt, t;      // ranges
};

// The producer's view of a piece: its keys.
struct Keys {
  int key0, end, row;     // ranges: first key, end of the keys; table row
  const int* list;        // lists: entries of the piece, `count` of them
  int count, seen;        // seen: keys before the token's own end
};

template <int D, bool kList>
__global__ void __launch_bounds__(kThreads, 1)
    rows_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_qs,
                const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                const __grid_constant__ RowsParams p) {
  using L = Layout<D>;
  constexpr int NS = L::kSlots;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* sQ = smem;
  uint8_t* sRing = smem + L::kOffRing;
  Piece* pieces = reinterpret_cast<Piece*>(smem + L::kOffPiece);  // [slot][2]
  uint64_t* bar_full = reinterpret_cast<uint64_t*>(smem + L::kOffBar);  // [NS] ring slot holds its tile
  uint64_t* bar_empty = bar_full + NS;    // [NS] ring slot read
  uint64_t* bar_sfull = bar_empty + NS;   // [2] scores complete
  uint64_t* bar_pfull = bar_sfull + 2;    // [2] P written (4 warps)
  uint64_t* bar_odone = bar_pfull + 2;    // [2] a piece's last P V complete
  uint64_t* bar_ofree = bar_odone + 2;    // [2] a piece's O read (4 warps)
  uint64_t* bar_qfull = bar_ofree + 2;    // [slot][2] rows loaded
  uint64_t* bar_qfree = bar_qfull + 4;    // [slot][2] a piece's last Q K^T complete
  uint64_t* bar_pieced = bar_qfree + 4;   // [slot][2] piece told
  uint64_t* bar_unpieced = bar_pieced + 4;  // [slot][2] piece done with (MMA thread, 4 warps)
  uint64_t* bar_fixset = bar_unpieced + 4;  // [4] clearing asked for
  uint64_t* bar_fixdone = bar_fixset + 4;   // [4] done
  uint64_t* bar_raw = bar_fixdone + 4;      // [4] value tile to be cleared landed
  uint64_t* bar_drain = bar_raw + 4;        // after an abort: the MMAs issued so far completed
  Fix* fixes = reinterpret_cast<Fix*>(smem + L::kOffFix);
  Plan* plan = reinterpret_cast<Plan*>(smem + L::kOffPlan);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kOffMisc + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = p.Hq / p.Hkv;

  if (threadIdx.x == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(bar_full + i, 1);
      mbar_init(bar_empty + i, 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar_sfull + s, 1);
      mbar_init(bar_pfull + s, 4);
      mbar_init(bar_odone + s, 1);
      mbar_init(bar_ofree + s, 4);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(bar_qfull + i, 1);
      mbar_init(bar_qfree + i, 1);
      mbar_init(bar_pieced + i, 1);
      mbar_init(bar_unpieced + i, 5);
      mbar_init(bar_fixset + i, 1);
      mbar_init(bar_fixdone + i, 1);
      mbar_init(bar_raw + i, 1);
    }
    mbar_init(bar_drain, 1);
    *abort_flag = 0;
    mbar_fence_init();
  }
  grid_depends();
  if (warp == 1) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  if (!kList)
    make_plan(p, plan, reinterpret_cast<long long*>(smem + L::kOffScan),
              reinterpret_cast<int*>(smem + L::kOffScan + 12 * 8));
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    // ---------------------------------------------------------------- producer
    const int cap = p.max_blocks * p.page_size;
    uint32_t ring = 0, fix_n = 0;
    uint32_t told[2] = {0, 0};
    uint32_t q_uses[2][2] = {{0, 0}, {0, 0}};
    // the last loads: whether on a ring slot's bar_full (its phase), on a bar_raw (its phase)
    uint32_t on_full = 0, full_ph = 0, on_raw = 0, raw_ph = 0;
    bool ok = true;

    // pages of 32 blocks of a piece, one a lane: number, row of the page; flags: bit 0 seen, bit 1 seen whole
    int pg[2], prow[2];
    uint32_t batch_seen[2] = {0, 0}, batch_full[2] = {0, 0};
    int batch_part[2] = {0, 0};
    Keys keys[2];

    auto page_of = [&](int row, int blk, int* out_row) {
      const int at = blk * 64 / p.page_size;
      int g = p.block_table[static_cast<long long>(row) * p.max_blocks + at];
      if (g < 0 || g >= p.num_pages) {
        record(2, kDevBadPage);
        g = 0;
      }
      *out_row = blk * 64 - at * p.page_size;
      return g;
    };
    // looks up blocks 32 i .. 32 i + 31 of slot s's piece
    auto look_up = [&](int s, int i) {
      const Keys& k = keys[s];
      bool seen = false;
      pg[s] = prow[s] = 0;
      int v = 0;
      if (kList) {
        const int e = 32 * i + lane;
        const int blk = e < k.count ? k.list[e] : -1;
        if (blk >= 0) {
          if (blk >= cap / 64)
            record(3, kDevBadPage);
          else
            v = min(64, k.seen - blk * 64);
        }
        seen = v > 0;
        if (seen) pg[s] = page_of(k.row, blk, &prow[s]);
      } else {
        const int key = k.key0 + 64 * (32 * i + lane);
        v = min(64, k.end - key);
        seen = v > 0;
        if (seen) pg[s] = page_of(k.row, key / 64, &prow[s]);
      }
      batch_seen[s] = __ballot_sync(0xffffffffu, seen);
      batch_full[s] = __ballot_sync(0xffffffffu, v == 64);
      const uint32_t some = batch_seen[s] & ~batch_full[s];
      batch_part[s] = some ? __shfl_sync(0xffffffffu, v, __ffs(some) - 1) : 0;  // the same for all of them
    };
    // loads the K or V tile j of slot s's piece into the next ring slot
    auto load = [&](int s, int j, bool is_v) {
      const int e = 2 * (j & 15);
      const int g0 = __shfl_sync(0xffffffffu, pg[s], e), g1 = __shfl_sync(0xffffffffu, pg[s], e + 1);
      const int r0 = __shfl_sync(0xffffffffu, prow[s], e), r1 = __shfl_sync(0xffffffffu, prow[s], e + 1);
      const bool s0 = batch_seen[s] >> e & 1u, s1 = batch_seen[s] >> (e + 1) & 1u;
      const bool f0 = batch_full[s] >> e & 1u, f1 = batch_full[s] >> (e + 1) & 1u;
      bool good = true;
      if (lane == 0) {
        const uint32_t slot = ring % NS;
        good = ring < NS || wait_one(bar_empty + slot, (ring / NS - 1) & 1, abort_flag, 11);
        const bool fix = is_v && !(f0 && f1);
        const uint32_t fi = fix_n & 3;
        if (good && fix && fix_n >= 4) good = wait_one(bar_fixdone + fi, (fix_n / 4 - 1) & 1, abort_flag, 12);
        if (good) {
          uint64_t* done = fix ? bar_raw + fi : bar_full + slot;
          const uint32_t bytes = (s0 ? L::kTile / 2 : 0) + (s1 ? L::kTile / 2 : 0);
          if (fix) {
            fixes[fi].slot = static_cast<int>(slot);
            fixes[fi].v0 = f0 ? 64 : (s0 ? batch_part[s] : 0);
            fixes[fi].v1 = f1 ? 64 : (s1 ? batch_part[s] : 0);
          }
          if (bytes)
            mbar_arrive_expect_tx(done, bytes);
          else
            mbar_arrive(done);
          const int h = pieces[s * 2 + ((told[s] - 1) & 1)].h;
          uint8_t* dst = sRing + slot * L::kTile;
          const CUtensorMap* tm = is_v ? &tm_v : &tm_k;
          for (int c = 0; c < D / 64; ++c) {
            if (s0) tma_load_4d(dst + c * L::kHalf, tm, done, c * 64, h, r0, g0);
            if (s1) tma_load_4d(dst + c * L::kHalf + 64 * 128, tm, done, c * 64, h, r1, g1);
          }
          if (fix) {
            mbar_arrive(bar_fixset + fi);
            on_full &= ~(1u << slot);
            on_raw |= 1u << fi;
            raw_ph = (raw_ph & ~(1u << fi)) | ((fix_n / 4 & 1u) << fi);
          } else {
            on_full |= 1u << slot;
            full_ph = (full_ph & ~(1u << slot)) | ((ring / NS & 1u) << slot);
          }
        }
        if (fix) ++fix_n;
      }
      ++ring;
      return __shfl_sync(0xffffffffu, static_cast<int>(good), 0) != 0;
    };
    // tells slot s's warps of its next piece; its masks are in place but for n = -1
    auto tell = [&](int s, int n, int share, int h, int tok0, int ntok, int dst) {
      bool good = true;
      if (lane == 0) {
        Piece& d = pieces[s * 2 + (told[s] & 1)];
        d.n = n;
        d.share = share;
        d.h = h;
        d.tok0 = tok0;
        d.ntok = ntok;
        d.key0 = keys[share ? 0 : s].key0;
        d.keys = keys[share ? 0 : s].end - d.key0;
        d.dst = dst;
        mbar_arrive(bar_pieced + s * 2 + (told[s] & 1));
      }
      ++told[s];
      return good;
    };
    // the place of slot s's next piece is free
    auto piece_free = [&](int s) {
      bool good = true;
      if (lane == 0 && told[s] >= 2)
        good = wait_one(bar_unpieced + s * 2 + (told[s] & 1), (told[s] / 2 - 1) & 1, abort_flag, 13);
      return __shfl_sync(0xffffffffu, static_cast<int>(good), 0) != 0;
    };
    // loads slot s's rows
    auto load_rows = [&](int s, int buf, bool pair, int h, int tok0) {
      bool good = true;
      if (lane == 0) {
        uint32_t& uses = q_uses[s][buf];
        if (uses > 0) good = wait_one(bar_qfree + s * 2 + buf, (uses - 1) & 1, abort_flag, 14);
        if (good) {
          const int tokens = pair ? p.tile_tokens : p.unit_tokens;
          mbar_arrive_expect_tx(bar_qfull + s * 2 + buf, static_cast<uint32_t>(tokens * G * D * 2));
          for (int c = 0; c < D / 64; ++c)
            tma_load_4d(sQ + s * L::kTile + c * L::kHalf + buf * (64 * 128), pair ? &tm_q : &tm_qs,
                        bar_qfull + s * 2 + buf, c * 64, 0, h, tok0);
          ++uses;
        }
      }
      return __shfl_sync(0xffffffffu, static_cast<int>(good), 0) != 0;
    };

    if (lane == 0) {
      tma_prefetch_desc(&tm_q);
      tma_prefetch_desc(&tm_qs);
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
    }
    bool pend_pair = false;
    int pend_j = 0;
    if (!kList && plan->pair_total > 0) {
      const int nt = tiles_of(plan->prefix_end);
      const int grid = gridDim.x;
      long long at = run_start(plan->pair_total, grid, blockIdx.x);
      const long long end = run_start(plan->pair_total, grid, blockIdx.x + 1);
      const int tokens = p.B * p.Nq;
      while (ok && at < end) {
        const int unit = static_cast<int>(at / nt), t = static_cast<int>(at - static_cast<long long>(unit) * nt);
        const int n = static_cast<int>(min(static_cast<long long>(nt - t), end - at));
        const int h = unit / p.pairs, pair = unit - h * p.pairs;
        // the last tile of the piece before goes in front of this one's rows
        if (pend_pair) ok = load(0, pend_j, true);
        pend_pair = false;
        keys[0].key0 = 128 * t;
        keys[0].end = plan->prefix_end;
        keys[0].row = 0;
        const int tok0 = 2 * pair * p.tile_tokens, tok1 = tok0 + p.tile_tokens;
        const int share = tok1 < tokens ? 1 : 2;
        for (int s = 0; ok && s < 2; ++s) {
          const int tok = s ? tok1 : tok0;
          ok = piece_free(s);
          if (ok) tell(s, n, share, h, tok, max(0, min(p.tile_tokens, tokens - tok)), static_cast<int>(blockIdx.x) + unit);
          if (ok && (s == 0 || share == 1)) ok = load_rows(s, 0, true, h, tok);
        }
        for (int j = 0; ok && j < n; ++j) {
          if (j > 0) ok = load(0, j - 1, true);
          if (ok && (j & 15) == 0) look_up(0, j >> 4);
          if (ok) ok = load(0, j, false);
        }
        pend_pair = true;
        pend_j = n - 1;
        at += n;
      }
    }
    // lanes
    Lane ln[2];
    int j[2] = {0, 0}, n[2] = {0, 0};
    bool fin[2] = {false, false}, pend[2] = {false, false};
    const int lanes = 2 * gridDim.x;
    const int units = p.B * p.Nq * p.Hkv, unit_tiles = (p.n_sel + 1) >> 1;  // lists
    const int whole = kList ? units / lanes * lanes : 0;
    const long long cut_total = static_cast<long long>(units - whole) * unit_tiles;
    for (int s = 0; s < 2; ++s) {
      const int l = lane_of(s);
      if (kList) {
        ln[s].unit = l;  // while below `whole`
        ln[s].left = run_start(cut_total, lanes, l + 1) - run_start(cut_total, lanes, l);
      } else {
        ln[s].left = run_start(plan->total, lanes, l + 1) - run_start(plan->total, lanes, l);
        if (ln[s].left > 0) {
          const int b = plan->lane_b[s];
          const int nt = b < 0 ? tiles_of(plan->prefix_end) : own_tiles(p, b);
          const long long at = plan->lane_at[s];
          const int u = static_cast<int>(at / nt), rt = b < 0 ? 1 : p.own_rt;
          ln[s].b = b;
          ln[s].h = u / rt;
          ln[s].rt = u - ln[s].h * rt;
          ln[s].t = static_cast<int>(at - static_cast<long long>(u) * nt);
        }
      }
    }
    if (ok && p.q_buffers == 2 && lane == 0) {
      // the second buffer of rows lies over the lower half of a pair's rows
      for (int s = 0; ok && s < 2; ++s)
        if (q_uses[s][0] > 0) ok = wait_one(bar_qfree + s * 2, (q_uses[s][0] - 1) & 1, abort_flag, 14);
    }
    ok = __shfl_sync(0xffffffffu, static_cast<int>(ok), 0) != 0;
    uint32_t q_next[2] = {0, 0};

    // next piece of slot s: told, its rows on their way; n[s] = 0 where there is none or nothing to compute
    auto next_piece = [&](int s) {
      Lane& w = ln[s];
      const int l = lane_of(s);
      Keys& k = keys[s];
      int h, tok0, ntok, dst;
      if (!piece_free(s)) return false;
      if (kList) {
        long long u;
        int t0 = 0, nt = unit_tiles;
        dst = -1;
        if (w.unit < whole) {
          u = w.unit;
          w.unit += lanes;
        } else if (w.left > 0) {
          const long long first = run_start(cut_total, lanes, l), at = run_start(cut_total, lanes, l + 1) - w.left;
          const int cu = static_cast<int>(at / unit_tiles);
          u = whole + cu;
          t0 = static_cast<int>(at - static_cast<long long>(cu) * unit_tiles);
          nt = static_cast<int>(min(static_cast<long long>(unit_tiles - t0), w.left));
          if (nt < unit_tiles) dst = 2 * l + (at > first ? 1 : 0);
          w.left -= nt;
        } else {
          fin[s] = true;
          return tell(s, -1, 0, 0, 0, 0, 0);
        }
        // units by sequence, head, token: neighbours read the same head's keys
        const int per = p.Hkv * p.Nq;
        const int b = static_cast<int>(u / per), r = static_cast<int>(u - static_cast<long long>(b) * per);
        h = r / p.Nq;
        const int i = r - h * p.Nq;
        tok0 = b * p.Nq + i;
        ntok = 1;
        const int len = clamped_len(p, b);
        if (lane == 0 && h == 0 && i == 0 && t0 == 0 && len != p.seqlens[b]) record(1, kDevBadSeqlen);
        k.row = b;
        k.seen = max(0, len - p.Nq + i + 1);
        k.list = p.blocks + (static_cast<long long>(tok0) * p.Hkv + h) * p.n_sel + 2 * t0;
        k.count = min(p.n_sel - 2 * t0, 2 * nt);
        k.key0 = k.end = 0;
        // which of them are seen; the last one that is ends the piece
        Piece& d = pieces[s * 2 + (told[s] & 1)];
        int last = -1;
        for (int i32 = (k.count - 1) >> 5; i32 >= 0; --i32) {  // ends with the first 32 looked up
          look_up(s, i32);
          if (lane == 0) {
            d.full[i32] = batch_full[s];
            d.some[i32] = batch_seen[s] & ~batch_full[s];
            if (d.some[i32]) d.part = batch_part[s];
          }
          if (last < 0 && batch_seen[s]) last = 32 * i32 + 31 - __clz(batch_seen[s]);
        }
        n[s] = (last + 2) >> 1;
      } else {
        if (w.left == 0) {
          fin[s] = true;
          return tell(s, -1, 0, 0, 0, 0, 0);
        }
        while (w.b >= 0 && w.t == 0 && w.rt == 0 && w.h == 0 && own_tiles(p, w.b) == 0) ++w.b;
        int nt, rts, unit;
        h = w.h;
        if (w.b < 0) {
          nt = tiles_of(plan->prefix_end);
          rts = 1;
          unit = h;
          k.key0 = 128 * w.t;
          k.end = plan->prefix_end;
          k.row = 0;
          tok0 = 0;
          ntok = p.B * p.Nq;
        } else {
          nt = own_tiles(p, w.b);
          rts = p.own_rt;
          unit = (w.b * p.Hkv + h) * rts + w.rt + (p.pairs ? 0 : p.Hkv);
          k.key0 = p.shared_len + 128 * w.t;
          k.end = clamped_len(p, w.b);
          k.row = w.b;
          tok0 = w.b * p.Nq + w.rt * p.own_tokens;
          ntok = min(p.own_tokens, p.Nq - w.rt * p.own_tokens);
        }
        dst = l + unit;
        n[s] = static_cast<int>(min(static_cast<long long>(nt - w.t), w.left));
        w.left -= n[s];
        w.t += n[s];
        if (w.t == nt) {
          w.t = 0;
          if (++w.rt == rts) {
            w.rt = 0;
            if (++w.h == p.Hkv) {
              w.h = 0;
              ++w.b;
            }
          }
        }
      }
      j[s] = 0;
      tell(s, n[s], 0, h, tok0, ntok, dst);
      if (n[s] == 0) return true;
      const int buf = p.q_buffers == 2 ? static_cast<int>(q_next[s]++ & 1) : 0;
      if (!load_rows(s, buf, false, h, tok0)) return false;
      if (!kList) look_up(s, 0);
      return true;
    };

    if (ok && pend_pair) ok = load(0, pend_j, true);
    while (ok && !(fin[0] && fin[1] && !pend[0] && !pend[1])) {
      for (int s = 0; ok && s < 2; ++s) {
        if (pend[s]) ok = load(s, j[s] - 1, true);
        pend[s] = false;
        while (ok && !fin[s] && j[s] == n[s]) ok = next_piece(s);
        if (ok && !fin[s]) {
          if (j[s] > 0 && (j[s] & 15) == 0) look_up(s, j[s] >> 4);
          ok = load(s, j[s], false);
          ++j[s];
          pend[s] = true;
        }
      }
    }
    if (ok && lane == 0) {
      // no more to clear
      const uint32_t fi = fix_n & 3;
      if (fix_n < 4 || wait_one(bar_fixdone + fi, (fix_n / 4 - 1) & 1, abort_flag, 12)) {
        fixes[fi].slot = -1;
        mbar_arrive(bar_fixset + fi);
      }
    }
    if (lane == 0) {
      // every load lands before the CTA may exit, whatever became of the others (bounded, not abortable)
      volatile int no_abort = 0;
      for (int i = 0; i < 4; ++i) {
        const uint32_t uses = q_uses[i >> 1][i & 1];
        if (uses > 0) mbar_wait(bar_qfull + i, (uses - 1) & 1, &no_abort, kWaitLimitNs);
        if (on_raw >> i & 1u) mbar_wait(bar_raw + i, raw_ph >> i & 1u, &no_abort, kWaitLimitNs);
      }
      for (int i = 0; i < NS; ++i)
        if (on_full >> i & 1u) mbar_wait(bar_full + i, full_ph >> i & 1u, &no_abort, kWaitLimitNs);
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer
    if (lane == 0) {
      constexpr uint32_t idesc_qk = idesc_bf16_f32(128, 128, 0);
      constexpr uint32_t idesc_pv = idesc_bf16_f32(128, D, 1);
      const uint64_t dQ = sdesc_sw128(smem_u32(sQ), 16, 1024);
      const uint64_t dK = sdesc_sw128(smem_u32(sRing), 16, 1024);
      const uint64_t dV = sdesc_sw128(smem_u32(sRing), L::kHalf, 1024);
      uint32_t ring = 0;
      uint32_t seen[2] = {0, 0};          // pieces looked at
      uint32_t done[2] = {0, 0};          // pieces with products
      uint32_t tiles[2] = {0, 0};         // P tiles consumed
      uint32_t q_uses[2][2] = {{0, 0}, {0, 0}};
      uint32_t q_lane[2] = {0, 0};
      int n[2] = {0, 0}, j[2] = {0, 0}, share[2] = {0, 0}, buf[2] = {0, 0};
      bool fin[2] = {false, false};
      bool pend[2] = {false, false}, pend_first[2] = {false, false}, pend_last[2] = {false, false};
      int pend_share[2] = {0, 0};
      uint32_t v_at = 0, k_at = 0;  // ring items that slot 1 shares
      bool ok = true;
      while (ok && !(fin[0] && fin[1] && !pend[0] && !pend[1])) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          if (!ok) break;
          const uint32_t tS = tmem + s * 128, tO = tmem + 256 + s * 128;
          if (pend[s]) {
            const bool shared = pend_share[s] != 0;
            const bool mine = !(s == 1 && pend_share[s] == 2);  // rows at all
            if (!(shared && s == 1)) v_at = ring++;
            const uint32_t vs = v_at % NS;
            if (mine) {
              if (!wait_one(bar_full + vs, (v_at / NS) & 1, abort_flag, 21) ||
                  !wait_one(bar_pfull + s, tiles[s] & 1, abort_flag, 22) ||
                  (pend_first[s] && done[s] > 0 && !wait_one(bar_ofree + s, (done[s] - 1) & 1, abort_flag, 23))) {
                ok = false;
                break;
              }
              ++tiles[s];
              tc_fence_after();
              const uint64_t dv = dV + static_cast<uint64_t>((vs * L::kTile) >> 4);
#pragma unroll
              for (int kk = 0; kk < 8; ++kk)
                mma_bf16_ts(tO, tS + kk * 8, dv + ((kk * 16 * 128) >> 4), idesc_pv, (!pend_first[s] || kk > 0) ? 1u : 0u);
              if (pend_last[s]) {
                mma_commit(bar_odone + s);
                ++done[s];
              }
              if (!(s == 0 && pend_share[s] == 1)) mma_commit(bar_empty + vs);
            }
            pend[s] = false;
          }
          while (!fin[s] && j[s] == n[s]) {
            uint64_t* told = bar_pieced + s * 2 + (seen[s] & 1);
            if (!wait_one(told, (seen[s] / 2) & 1, abort_flag, 24)) {
              ok = false;
              break;
            }
            const volatile Piece& d = pieces[s * 2 + (seen[s] & 1)];
            const int dn = d.n;
            share[s] = d.share;
            mbar_arrive(bar_unpieced + s * 2 + (seen[s] & 1));
            ++seen[s];
            fin[s] = dn < 0;
            n[s] = max(dn, 0);
            j[s] = 0;
            if (n[s] > 0) buf[s] = share[s] == 0 && p.q_buffers == 2 ? static_cast<int>(q_lane[s]++ & 1) : 0;
          }
          if (!ok) break;
          if (fin[s]) continue;
          const bool shared = share[s] != 0, mine = !(s == 1 && share[s] == 2);
          if (!(shared && s == 1)) k_at = ring++;
          const uint32_t ks = k_at % NS;
          if (mine) {
            const int qb = s * 2 + buf[s];
            if (!wait_one(bar_full + ks, (k_at / NS) & 1, abort_flag, 25) ||
                (j[s] == 0 && !wait_one(bar_qfull + qb, q_uses[s][buf[s]] & 1, abort_flag, 26))) {
              ok = false;
              break;
            }
            if (j[s] == 0) ++q_uses[s][buf[s]];
            tc_fence_after();
            const uint64_t da = dQ + static_cast<uint64_t>((s * L::kTile + buf[s] * (64 * 128)) >> 4);
            const uint64_t db = dK + static_cast<uint64_t>((ks * L::kTile) >> 4);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t off = ((kk >> 2) * L::kHalf + (kk & 3) * 32) >> 4;
              mma_bf16_ss(tS, da + off, db + off, idesc_qk, kk > 0 ? 1u : 0u);
            }
            mma_commit(bar_sfull + s);
            if (j[s] == n[s] - 1) mma_commit(bar_qfree + qb);
            if (!(s == 0 && share[s] == 1)) mma_commit(bar_empty + ks);
          }
          pend[s] = mine;
          pend_first[s] = j[s] == 0;
          pend_share[s] = share[s];
          ++j[s];
          pend_last[s] = j[s] == n[s];
        }
      }
      if (!ok) {
        // the MMAs issued so far complete before TMEM is freed
        volatile int no_abort = 0;
        mma_commit(bar_drain);
        mbar_wait(bar_drain, 0, &no_abort, kWaitLimitNs);
      }
    }
  } else if (warp == 2) {
    // ---------------------------------------------------------------- clearing
    // Value rows behind the keys that count hold anything, NaN included, and
    // P = 0 times NaN is not 0; halves that were not loaded hold older tiles.
    for (uint32_t i = 0;; ++i) {
      const uint32_t fi = i & 3;
      if (!wait_all(bar_fixset + fi, (i / 4) & 1, abort_flag, 31)) break;
      const int slot = fixes[fi].slot, v0 = fixes[fi].v0, v1 = fixes[fi].v1;
      if (slot < 0) break;
      if (!wait_all(bar_raw + fi, (i / 4) & 1, abort_flag, 32)) break;
      uint8_t* base = sRing + slot * L::kTile;
      for (int c = 0; c < D / 64; ++c)
        for (int half = 0; half < 2; ++half) {
          const int v = half ? v1 : v0;
          for (int off = v * 128 + lane * 16; off < 64 * 128; off += 512)
            *reinterpret_cast<uint4*>(base + c * L::kHalf + half * (64 * 128) + off) = make_uint4(0u, 0u, 0u, 0u);
        }
      fence_proxy_async_smem();  // these stores before the tensor core's reads
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar_full + slot);
        mbar_arrive(bar_fixdone + fi);
      }
    }
  } else if (warp >= 4) {
    // ---------------------------------------------------------------- softmax and results
    const int s = (warp - 4) >> 2, quarter = warp & 3;
    const int r = quarter * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t tS = tmem + s * 128 + lane_off, tO = tmem + 256 + s * 128 + lane_off;
    const int rtok = r / G, rg = r - rtok * G;
    uint32_t tiles = 0, done = 0;
    bool ok = true;
    for (uint32_t i = 0; ok; ++i) {
      const Piece& d = pieces[s * 2 + (i & 1)];
      if (!wait_all(bar_pieced + s * 2 + (i & 1), (i / 2) & 1, abort_flag, 41)) break;
      const int n = d.n, share = d.share, ntok = d.ntok, h = d.h, dst = d.dst;
      const int rows = share == 2 && s == 1 ? 0 : ntok * G;
      const bool live = r < rows;
      const int tok = d.tok0 + rtok;
      const int b = live ? tok / p.Nq : 0, nth = tok - b * p.Nq;
      if (n >= 0 && rows > 0) {
        // result rows, or a piece's
        float* part = nullptr;
        float* lse_part = nullptr;
        if (dst >= 0) {
          const long long at = share ? static_cast<long long>(dst) * 256 + s * 128 + r
                                     : p.pair_rows + static_cast<long long>(dst) * p.unit_rows + r;
          part = p.o_part + at * D;
          lse_part = p.lse_part + at;
        }
        __nv_bfloat16* orow = static_cast<__nv_bfloat16*>(p.o) + (static_cast<long long>(tok) * p.Hq + h * G + rg) * D;
        float* lrow = p.lse + (static_cast<long long>(b) * p.Hq + h * G + rg) * p.Nq + nth;
        float M = live ? -INFINITY : 0.f, l = 0.f;
        const float c = live ? p.scale_log2 : 0.f;
        if (n > 0) {
          // keys seen of the piece's
          const int lim = kList || !live ? 0 : min(d.keys, clamped_len(p, b) - p.Nq + nth + 1 - d.key0);
          for (int j = 0; j < n; ++j) {
            if (!wait_all(bar_sfull + s, tiles & 1, abort_flag, 42)) {
              ok = false;
              break;
            }
            ++tiles;
            tc_fence_after();
            if (quarter * 32 < rows) {
              Visible vis;
              bool whole;
              if (kList) {
                const int e = 2 * j;
                const uint32_t f = d.full[e >> 5] >> (e & 31), m = d.some[e >> 5] >> (e & 31);
                vis.v[0] = f & 1u ? 64 : (m & 1u ? d.part : 0);
                vis.v[1] = f & 2u ? 64 : (m & 2u ? d.part : 0);
                whole = (f & 3u) == 3u;
              } else {
                vis.v[0] = min(max(lim - 128 * j, 0), 64);
                vis.v[1] = min(max(lim - 128 * j - 64, 0), 64);
                whole = __all_sync(0xffffffffu, !live || vis.v[1] == 64);
              }
              RowTile t;
              if (__any_sync(0xffffffffu, M == -INFINITY))
                t = whole ? rows_first<false>(tS, vis, c, M) : rows_first<true>(tS, vis, c, M);
              else
                t = whole ? rows_tile<false>(tS, vis, c, M, live) : rows_tile<true>(tS, vis, c, M, live);
              const bool moved = live && t.M != M;
              const float a = !moved ? 1.f : (M == -INFINITY ? 0.f : ex2_approx(M - t.M));
              l = l * a + t.sum;
              if (j > 0 && __any_sync(0xffffffffu, moved && M != -INFINITY)) {
                // O holds the sum through the tile before: its P V completed before these scores were formed
                const float f = moved && M != -INFINITY ? a : 1.f;
                const float2 a2 = make_float2(f, f);
#pragma unroll
                for (int cc = 0; cc < D / 32; ++cc) {
                  uint32_t w[32];
                  tmem_ld32(tO + cc * 32, w);
                  tmem_wait_ld();
#pragma unroll
                  for (int x = 0; x < 16; ++x) {
                    const float2 y = fmul2(make_float2(__uint_as_float(w[2 * x]), __uint_as_float(w[2 * x + 1])), a2);
                    w[2 * x] = __float_as_uint(y.x);
                    w[2 * x + 1] = __float_as_uint(y.y);
                  }
                  tmem_st32(tO + cc * 32, w);
                }
              }
              M = live ? t.M : 0.f;
              tmem_wait_st();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_pfull + s);
          }
          if (!ok) break;
          if (!wait_all(bar_odone + s, done & 1, abort_flag, 43)) break;
          ++done;
          tc_fence_after();
        }
        // l is 0 where nothing was seen; NaN stays NaN
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const float lse2 = l == 0.f ? -INFINITY : M + __log2f(l);
        if (quarter * 32 < rows) {
#pragma unroll
          for (int cc = 0; cc < D / 32; ++cc) {
            uint32_t w[32];
            if (n > 0) {
              tmem_ld32(tO + cc * 32, w);
              tmem_wait_ld();
            }
#pragma unroll
            for (int x = 0; x < 32; ++x) w[x] = n > 0 && l != 0.f ? __float_as_uint(__uint_as_float(w[x]) * inv) : 0u;
            if (live) {
              if (dst >= 0) {
                uint4* to = reinterpret_cast<uint4*>(part + cc * 32);
#pragma unroll
                for (int x = 0; x < 8; ++x) to[x] = make_uint4(w[4 * x], w[4 * x + 1], w[4 * x + 2], w[4 * x + 3]);
              } else {
                uint4* to = reinterpret_cast<uint4*>(orow + cc * 32);
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                  uint32_t y[4];
#pragma unroll
                  for (int z = 0; z < 4; ++z)
                    y[z] = pack_bf16x2(__uint_as_float(w[8 * x + 2 * z]), __uint_as_float(w[8 * x + 2 * z + 1]));
                  to[x] = make_uint4(y[0], y[1], y[2], y[3]);
                }
              }
            }
          }
          if (live) {
            if (dst >= 0)
              *lse_part = lse2;
            else
              *lrow = lse2 * 0.6931471805599453f;
          }
        }
        if (n > 0) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar_ofree + s);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_unpieced + s * 2 + (i & 1));
      if (n < 0) break;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// ---------------------------------------------------------------------------
// Joining a row's pieces: LSE = log2 sum 2^LSE_i, O = sum 2^(LSE_i - LSE) O_i,
// in order.  A warp a row.
constexpr int kJoinWarps = 4;

struct Join {
  float m, l;
};
// Adds pieces first .. first + n - 1 (rows `row` of `rows` each, from `base` on) to a row's sums, which are kept
// under the largest LSE so far.
template <int D>
__device__ __forceinline__ void join(const RowsParams& p, long long base, long long first, int n, int rows, int row,
                                     Join& s, float (&acc)[D / 32]) {
  const int lane = threadIdx.x & 31;
  for (int i0 = 0; i0 < n; i0 += 32) {
    const int cnt = min(32, n - i0);
    const long long at = base + (first + i0) * rows + row;
    const float mine = lane < cnt ? p.lse_part[at + static_cast<long long>(lane) * rows] : -INFINITY;
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
    for (int x = 0; x < D / 32; ++x) acc[x] *= a;
#pragma unroll 4
    for (int i = 0; i < cnt; ++i) {
      const float wi = __shfl_sync(0xffffffffu, w, i);
      const float* o = p.o_part + (at + static_cast<long long>(i) * rows) * D + lane * (D / 32);
      s.l += wi;
      if (D == 128) {
        const float4 v = *reinterpret_cast<const float4*>(o);
        acc[0] = fmaf(wi, v.x, acc[0]);
        acc[1] = fmaf(wi, v.y, acc[1]);
        acc[D / 32 - 2] = fmaf(wi, v.z, acc[D / 32 - 2]);
        acc[D / 32 - 1] = fmaf(wi, v.w, acc[D / 32 - 1]);
      } else {
        const float2 v = *reinterpret_cast<const float2*>(o);
        acc[0] = fmaf(wi, v.x, acc[0]);
        acc[1] = fmaf(wi, v.y, acc[1]);
      }
    }
  }
}

template <int D>
__device__ __forceinline__ void write_row(const RowsParams& p, int tok, int hq, const Join& s, const float (&acc)[D / 32]) {
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

template <int D>
__global__ void __launch_bounds__(32 * kJoinWarps) join_ranges_kernel(const __grid_constant__ RowsParams p, int grid) {
  grid_depends();
  const int row = blockIdx.x * kJoinWarps + (threadIdx.x >> 5);
  if (row >= p.B * p.Nq * p.Hq) return;
  const int G = p.Hq / p.Hkv;
  const int tok = row / p.Hq, hq = row - tok * p.Hq, h = hq / G, g = hq - h * G;
  const int b = tok / p.Nq, i = tok - b * p.Nq;
  const long long total = p.sums[p.B], pair_total = p.sums[p.B + 1];
  const int nt = tiles_of(static_cast<int>(p.sums[p.B + 2]));
  Join s = {-INFINITY, 0.f};
  float acc[D / 32];
#pragma unroll
  for (int x = 0; x < D / 32; ++x) acc[x] = 0.f;
  if (p.pairs) {
    if (nt > 0) {
      const int rt = tok / p.tile_tokens, unit = h * p.pairs + (rt >> 1);
      const long long a = static_cast<long long>(unit) * nt;
      const int first = run_of(pair_total, grid, a), last = run_of(pair_total, grid, a + nt - 1);
      join<D>(p, 0, static_cast<long long>(first) + unit, last - first + 1, 256,
              (rt & 1) * 128 + (tok - rt * p.tile_tokens) * G + g, s, acc);
    }
  } else if (nt > 0) {
    const long long a = static_cast<long long>(h) * nt;
    const int first = run_of(total, 2 * grid, a), last = run_of(total, 2 * grid, a + nt - 1);
    join<D>(p, p.pair_rows, static_cast<long long>(first) + h, last - first + 1, p.unit_rows, tok * G + g, s, acc);
  }
  const int own = own_tiles(p, b);
  if (own > 0) {
    const int rt = i / p.own_tokens, u = h * p.own_rt + rt;
    const long long a = p.sums[b] + static_cast<long long>(u) * own;
    const int first = run_of(total, 2 * grid, a), last = run_of(total, 2 * grid, a + own - 1);
    const long long unit = static_cast<long long>(b) * p.Hkv * p.own_rt + u + (p.pairs ? 0 : p.Hkv);
    join<D>(p, p.pair_rows, first + unit, last - first + 1, p.unit_rows, (i - rt * p.own_tokens) * G + g, s, acc);
  }
  write_row<D>(p, tok, hq, s, acc);
}

// Units of listed blocks that more than one lane computed.
template <int D>
__global__ void __launch_bounds__(32 * kJoinWarps) join_lists_kernel(const __grid_constant__ RowsParams p, int grid) {
  grid_depends();
  const int G = p.Hq / p.Hkv, lanes = 2 * grid;
  const int units = p.B * p.Nq * p.Hkv, unit_tiles = (p.n_sel + 1) >> 1;
  const int whole = units / lanes * lanes;
  const long long total = static_cast<long long>(units - whole) * unit_tiles;
  const int r = blockIdx.x * kJoinWarps + (threadIdx.x >> 5);
  if (r >= (units - whole) * G) return;
  const int cu = r / G, g = r - cu * G;
  const long long a = static_cast<long long>(cu) * unit_tiles;
  const int first = run_of(total, lanes, a), last = run_of(total, lanes, a + unit_tiles - 1);
  if (first == last) return;  // written as it is
  Join s = {-INFINITY, 0.f};
  float acc[D / 32];
#pragma unroll
  for (int x = 0; x < D / 32; ++x) acc[x] = 0.f;
  // a lane's first piece, unless it started in the unit before
  const int second = run_start(total, lanes, first) < a ? 1 : 0;
  join<D>(p, 0, 2ll * first + second, 1, p.unit_rows, g, s, acc);
  // its place is 2 lane: every second piece from the next lane on
  for (int l = first + 1; l <= last; ++l) join<D>(p, 0, 2ll * l, 1, p.unit_rows, g, s, acc);
  const int per = p.Hkv * p.Nq, u = whole + cu;
  const int b = u / per, x = u - b * per, h = x / p.Nq;
  write_row<D>(p, b * p.Nq + x - h * p.Nq, h * G + g, s, acc);
}

template <int D>
cudaError_t launch_d(RowsParams p, const CUtensorMap& tm_q, const CUtensorMap& tm_qs, const CUtensorMap& tm_k,
                     const CUtensorMap& tm_v, cudaStream_t stream) {
  using L = Layout<D>;
  int dev = 0, n_sm = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  int grid = n_sm < kRowsCtas ? n_sm : kRowsCtas;
  const int G = p.Hq / p.Hkv;
  if (p.blocks) {
    const long long tiles = static_cast<long long>(p.B) * p.Nq * p.Hkv * ((p.n_sel + 1) / 2);
    if ((tiles + 1) / 2 < grid) grid = static_cast<int>((tiles + 1) / 2);
    auto kern = rows_kernel<D, true>;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kAlloc);
    if (e == cudaSuccess) e = launch_dependent(kern, dim3(grid), kThreads, L::kAlloc, stream, tm_q, tm_qs, tm_k, tm_v, p);
    if (e != cudaSuccess) return e;
    const int units = p.B * p.Nq * p.Hkv, cut = units - units / (2 * grid) * (2 * grid);
    if (cut == 0) return e;
    return launch_dependent(join_lists_kernel<D>, dim3((cut * G + kJoinWarps - 1) / kJoinWarps), 32 * kJoinWarps, 0,
                            stream, p, grid);
  }
  auto kern = rows_kernel<D, false>;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kAlloc);
  if (e == cudaSuccess) e = launch_dependent(kern, dim3(grid), kThreads, L::kAlloc, stream, tm_q, tm_qs, tm_k, tm_v, p);
  if (e != cudaSuccess) return e;
  const long long rows = static_cast<long long>(p.B) * p.Nq * p.Hq;
  return launch_dependent(join_ranges_kernel<D>, dim3(static_cast<unsigned>((rows + kJoinWarps - 1) / kJoinWarps)),
                          32 * kJoinWarps, 0, stream, p, grid);
}

}  // namespace

RowsSizes rows_sizes(int B, int Nq, int Hq, int Hkv, bool lists) {
  RowsSizes z;
  const int G = Hq / Hkv;
  const long long tokens = static_cast<long long>(B) * Nq;
  z.tile_tokens = 128 / G;
  z.pairs = 0;
  if (lists) {
    z.own_tokens = z.own_rt = z.unit_tokens = 1;
    z.pair_rows = 0;
    z.unit_rows = G;
    z.lane_pieces = 4ll * kRowsCtas;
  } else {
    const long long tiles = (tokens + z.tile_tokens - 1) / z.tile_tokens;
    if (tiles > 1) z.pairs = static_cast<int>((tiles + 1) / 2);
    z.own_tokens = Nq < z.tile_tokens ? Nq : z.tile_tokens;
    z.own_rt = (Nq + z.own_tokens - 1) / z.own_tokens;
    // without pairs a prefix' unit holds all tokens
    z.unit_tokens = z.pairs ? z.own_tokens : static_cast<int>(tokens);
    z.unit_rows = z.unit_tokens * G;
    z.pair_rows = z.pairs ? (kRowsCtas + static_cast<long long>(Hkv) * z.pairs) * 256 : 0;
    z.lane_pieces = 2ll * kRowsCtas + static_cast<long long>(B) * Hkv * z.own_rt + (z.pairs ? 0 : Hkv);
  }
  return z;
}

cudaError_t launch_rows(const RowsParams& p, const CUtensorMap& tm_q, const CUtensorMap& tm_qs, const CUtensorMap& tm_k,
                        const CUtensorMap& tm_v, cudaStream_t stream) {
  return p.d == 64 ? launch_d<64>(p, tm_q, tm_qs, tm_k, tm_v, stream)
                   : launch_d<128>(p, tm_q, tm_qs, tm_k, tm_v, stream);
}

cudaError_t status_word_rows(uint32_t** at) { return cudaGetSymbolAddress(reinterpret_cast<void**>(at), g_rows_status); }

}  // namespace attn

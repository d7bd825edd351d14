// Attention of many tokens over listed 64-key blocks of a paged bf16 cache, block
// by block, for sm_103a: where many of the tokens list a block, its keys and
// values are loaded once for all of them.
//
// Token by token (few_rows_sm103.cu) each list entry takes its block, 256 d bytes,
// from L2, and that bounds it: 2048 tokens on 32 blocks each, 8 KV heads of
// d = 128, are 17 GB and 1140 us.  Here the entries are sorted by (KV head, block);
// a tile is one block and the rows (token, head of the group) that list it, 128 at
// most:
//     S [128 x 64] = Q K^T,  O_i = softmax(S) V,  LSE_i.
// What an entry leaves, G rows of d + 1 fp32 (a piece), lies tile by tile, so that a
// tile is written by a few large boxes, and a second kernel joins the pieces of each
// row, 512 bytes at a time (d = 128).  That moves 8 G d bytes an entry, an eighth with
// G = 4, and bounds it: on the case above 1.2 GB in 236 us (5.2 TB/s) and 1.1 GB in
// 177 us (6.1 TB/s); sorting takes 35 us, the whole 472 us.
//
// Sorting: counts of the entries of each block, by atomics whose answer is the
// entry's place among them (the order of a tile's rows, on which no result
// depends: a row is what its query and the block make of it, and a row's pieces are
// joined in the order of its list); sums over the blocks, with the list of tiles; each
// entry's token to its place.
//
// The tokens of a sequence are cut into chunks whose pieces take 1 GB at most
// (the case above in chunks of 256 MB: 622 us, as each reads the blocks again and has
// fuller tiles the more tokens it has).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "launch.h"
#include "ptx.cuh"
#include "rows_join.cuh"
#include "rows_plan.cuh"

namespace attn {
namespace {

__device__ __forceinline__ int length_of(const ByBlockParams& p, int b) {
  return min(max(p.seqlens[b], 0), p.max_blocks * p.page_size);
}
// Whether one of two bf16 is infinite or not a number.
__device__ __forceinline__ bool not_finite(uint32_t x) {
  return (x & 0x7f80u) == 0x7f80u || (x & 0x7f800000u) == 0x7f800000u;
}
// Keys that token i of sequence b sees.
__device__ __forceinline__ int seen_by(const ByBlockParams& p, int b, int i) { return max(0, length_of(p, b) - p.Nq + i + 1); }

// ---------------------------------------------------------------------------
// Sorting.  A warp a list.
constexpr int kSortWarps = 8;

struct ListAt {
  int tok, h, b, i, chunk, seen;
  const int* list;
  long long entry;  // first of its entries
  long long block0;  // first of the blocks of its sequence, chunk and KV head
};
__device__ __forceinline__ bool list_at(const ByBlockParams& p, ListAt& l) {
  const long long w = static_cast<long long>(blockIdx.x) * kSortWarps + (threadIdx.x >> 5);
  if (w >= static_cast<long long>(p.B) * p.Nq * p.Hkv) return false;
  l.tok = static_cast<int>(w / p.Hkv);
  l.h = static_cast<int>(w - static_cast<long long>(l.tok) * p.Hkv);
  l.b = l.tok / p.Nq;
  l.i = l.tok - l.b * p.Nq;
  l.chunk = l.i / p.chunk_tokens;
  l.seen = seen_by(p, l.b, l.i);
  l.entry = w * p.n_sel;
  l.list = p.blocks + l.entry;
  l.block0 = (static_cast<long long>(l.b * p.chunks + l.chunk) * p.Hkv + l.h) * p.n_blocks;
  return true;
}

__global__ void __launch_bounds__(32 * kSortWarps) count_kernel(const __grid_constant__ ByBlockParams p) {
  ListAt l;
  if (!list_at(p, l)) return;
  const int lane = threadIdx.x & 31;
  if (lane == 0 && l.h == 0 && l.i == 0 && length_of(p, l.b) != p.seqlens[l.b]) record(1, kDevBadSeqlen);
  for (int s = lane; s < p.n_sel; s += 32) {
    const int blk = l.list[s];
    if (blk >= p.n_blocks) record(3, kDevBadPage);
    if (blk >= 0 && blk < p.n_blocks && blk * 64 < l.seen) p.rank[l.entry + s] = atomicAdd(p.counts + l.block0 + blk, 1);
  }
}

// Counts to starts, and the tiles: a CTA a chunk and KV head, which adds up what the heads before it have.
constexpr int kPlanThreads = 1024;
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const __grid_constant__ ByBlockParams p) {
  grid_depends();
  __shared__ unsigned long long s_sum[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int group = blockIdx.x / p.Hkv, h = blockIdx.x - group * p.Hkv, b = group / p.chunks;
  const int n = p.n_blocks, first_j = h * n;
  const int* counts = p.counts + static_cast<long long>(group) * p.Hkv * n;
  int2* starts = p.starts + static_cast<long long>(group) * p.Hkv * n;
  int4* tiles = p.tiles + static_cast<long long>(group) * p.tile_cap;
  // tiles, and in the upper half 32's of rows: full tiles take 128, the last one what it needs
  const int G = p.Hq / p.Hkv;
  auto packed = [&](int c) {
    const int full = c / p.tile_tokens, rest = c - full * p.tile_tokens;
    return static_cast<unsigned long long>(4 * full + (rest * G + 31) / 32) << 32 | static_cast<unsigned>(full + (rest > 0 ? 1 : 0));
  };
  unsigned long long base = 0;
  for (int j = tid; j < first_j; j += kPlanThreads) base += packed(counts[j]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) base += __shfl_xor_sync(0xffffffffu, base, o);
  if (lane == 0) s_sum[warp] = base;
  __syncthreads();
  base = s_sum[lane];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) base += __shfl_xor_sync(0xffffffffu, base, o);
  for (int j0 = 0; j0 < n; j0 += kPlanThreads) {
    const int blk = j0 + tid, j = first_j + blk, c = blk < n ? counts[j] : 0;
    const unsigned long long mine = packed(c);
    unsigned long long sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long y = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += y;
    }
    __syncthreads();
    if (lane == 31) s_sum[warp] = sum;
    __syncthreads();
    unsigned long long w = s_sum[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    const unsigned long long before = base + sum - mine + (warp ? __shfl_sync(0xffffffffu, w, warp - 1) : 0);
    base += __shfl_sync(0xffffffffu, w, 31);
    if (c > 0) {
      const int first = static_cast<int>(before), rows = static_cast<int>(before >> 32);
      const int at_page = blk * 64 / p.page_size;
      int g = p.block_table[static_cast<long long>(b) * p.max_blocks + at_page];
      if (g < 0 || g >= p.num_pages) {
        record(2, kDevBadPage);
        g = 0;
      }
      g = g * (p.page_size / 8) + 8 * (blk - at_page * (p.page_size / 64));
      starts[j] = make_int2(first, rows);
      for (int k = 0; k * p.tile_tokens < c; ++k)
        tiles[first + k] = make_int4(j, rows + 4 * k, min(p.tile_tokens, c - k * p.tile_tokens), g);
    }
  }
  if (tid == 0 && h == p.Hkv - 1) p.n_tiles[group] = static_cast<int>(base);
}

// order: the tokens of the chunk that list a block, tile after tile.
__global__ void __launch_bounds__(32 * kSortWarps) place_kernel(const __grid_constant__ ByBlockParams p) {
  grid_depends();
  ListAt l;
  if (!list_at(p, l)) return;
  const int i0 = l.chunk * p.chunk_tokens;
  int* order = p.order + static_cast<long long>(l.b * p.chunks + l.chunk) * p.tile_cap * p.tile_tokens;
  for (int s = threadIdx.x & 31; s < p.n_sel; s += 32) {
    const int blk = l.list[s];
    if (blk >= 0 && blk < p.n_blocks && blk * 64 < l.seen)
      order[static_cast<long long>(p.starts[l.block0 + blk].x) * p.tile_tokens + p.rank[l.entry + s]] = l.i - i0;
  }
}

// ---------------------------------------------------------------------------
// Attention of one chunk's tiles, dealt to the CTAs in equal runs.
//
// Warps: 0 loader of blocks, 1 issuer, 2 and 3 gather the rows' queries, 4-7 and
// 8-11 softmax and results of even and odd tiles.
constexpr int kThreads = 384;
constexpr int kNotes = 8;  // blocks with notes of values that are not finite: more than can be between loading and results

template <int D>
struct Layout {
  static constexpr int kGroup = D / 64 * 1024;
  static constexpr int kBlock = 64 * D * 2;   // K or V of a block
  static constexpr int kHalf = 128 * 128;     // 64 columns of 128 rows
  static constexpr int kQ = 128 * D * 2;
  static constexpr int kQs = 2, kKvs = 3;
  static constexpr int kOut = 32 * 128;       // outputs on their way to memory: 32 columns of a warp's rows, twice
  static constexpr int kOffKv = kQs * kQ;
  static constexpr int kOffOut = kOffKv + kKvs * 2 * kBlock;
  static constexpr int kOffBar = kOffOut + 8 * 2 * kOut;
  static constexpr int kNumBars = 2 * kQs + 2 * kKvs + 4 * 2 + 2;
  static constexpr int kOffNote = kOffBar + 8 * kNumBars;  // [kNotes][D] first key with a value that is not finite
  static constexpr int kOffNoted = kOffNote + kNotes * D;  // [kNotes]
  static constexpr int kOffMisc = kOffNoted + kNotes * 4;
  static constexpr int kBytes = kOffMisc + 16;
  static constexpr int kAlloc = kBytes + 1024;
  static constexpr uint32_t kTmem = D == 64 ? 256 : 512;  // S twice, O twice
};
static_assert(Layout<128>::kAlloc <= 232448 && Layout<64>::kAlloc <= 232448, "shared memory of a CTA");

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    by_block_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                    const __grid_constant__ CUtensorMap tm_o, const __grid_constant__ ByBlockParams p, int group) {
  using L = Layout<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t *sm_q = smem, *sm_kv = smem + L::kOffKv;
  uint64_t* qfull = reinterpret_cast<uint64_t*>(smem + L::kOffBar);  // queries there (2 warps)
  uint64_t* qempty = qfull + L::kQs;      // read
  uint64_t* kvfull = qempty + L::kQs;     // block there
  uint64_t* kvempty = kvfull + L::kKvs;   // read
  uint64_t* sfull = kvempty + L::kKvs;    // [2] scores complete
  uint64_t* pfull = sfull + 2;            // [2] P written (4 warps)
  uint64_t* odone = pfull + 2;            // [2] P V complete
  uint64_t* ofree = odone + 2;            // [2] O read (4 warps)
  uint64_t* raw = ofree + 2;              // a block to be looked through landed
  uint64_t* drain = raw + 1;              // after an abort: the MMAs issued so far completed
  uint8_t* note = smem + L::kOffNote;
  volatile int* noted = reinterpret_cast<volatile int*>(smem + L::kOffNoted);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kOffMisc + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < L::kQs; ++i) {
      mbar_init(qfull + i, 2);
      mbar_init(qempty + i, 1);
    }
    for (int i = 0; i < L::kKvs; ++i) {
      mbar_init(kvfull + i, 1);
      mbar_init(kvempty + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(sfull + i, 1);
      mbar_init(pfull + i, 4);
      mbar_init(odone + i, 1);
      mbar_init(ofree + i, 4);
    }
    mbar_init(raw, 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    mbar_fence_init();
  }
  grid_depends();
  if (warp == 1) {
    tmem_alloc(tmem_slot, L::kTmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  const int G = p.Hq / p.Hkv;
  const int b = group / p.chunks, i0 = (group - b * p.chunks) * p.chunk_tokens;
  const long long tok0 = static_cast<long long>(b) * p.Nq + i0;
  const long long total = p.n_tiles[group];
  const int x0 = static_cast<int>(run_start(total, gridDim.x, blockIdx.x));
  const int n = static_cast<int>(run_start(total, gridDim.x, blockIdx.x + 1)) - x0;
  const int4* tiles = p.tiles + static_cast<long long>(group) * p.tile_cap + x0;
  const int* order = p.order + (static_cast<long long>(group) * p.tile_cap + x0) * p.tile_tokens;
  const int len = length_of(p, b), first_seen = len - p.Nq + i0 + 1;  // keys of all, of the first token (below 1: none)

  if (warp == 0) {
    if (lane == 0) {
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
    }
    int cur = -1;
    uint32_t kv = 0, raws = 0;
    bool ok = true;
    int4 t = n > 0 ? tiles[0] : make_int4(-1, 0, 0, 0);
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      const int4 next = i + 1 < n ? tiles[i + 1] : t;
      if (t.x != cur) {
        cur = t.x;
        const int h = cur / p.n_blocks, key0 = 64 * (cur - h * p.n_blocks);
        const uint32_t slot = kv % L::kKvs;
        if (kv >= L::kKvs) ok = wait_all(kvempty + slot, (kv / L::kKvs - 1) & 1, abort_flag, 11);
        if (!ok) break;
        uint8_t* at = sm_kv + slot * 2 * L::kBlock;
        // whether some row does not see all of the block's values
        const bool part = key0 + 64 > first_seen;
        uint64_t* full = part ? raw : kvfull + slot;
        if (lane == 0) {
          if (!part) noted[kv % kNotes] = 0;
          mbar_arrive_expect_tx(full, 2 * L::kBlock);
          tma_load_5d(at, &tm_k, full, 0, 0, 0, t.w, h);
          tma_load_5d(at + L::kBlock, &tm_v, full, 0, 0, 0, t.w, h);
        }
        if (part) {
          // behind the sequence's end there may be anything: cleared.  A value that is not finite and that some of
          // the rows do not see is cleared too (0 times it is NaN) and noted: the results of those that see it get it
          volatile int no_abort = 0;
          ok = mbar_wait(raw, raws++ & 1, &no_abort, kWaitLimitNs);
          if (!ok) record(12, kDevTimeout);
          if (!__all_sync(0xffffffffu, ok)) {
            *abort_flag = 1;
            ok = false;
            break;
          }
          uint8_t* v = at + L::kBlock;
          if (key0 + 64 > len) {
            for (int c = lane; c < (key0 + 64 - len) * (D / 8); c += 32) {
              const int r = len - key0 + c / (D / 8), ch = c % (D / 8);
              *reinterpret_cast<uint4*>(v + (r >> 3) * L::kGroup + (ch >> 3) * 1024 + (r & 7) * 128 + (ch & 7) * 16) =
                  make_uint4(0u, 0u, 0u, 0u);
            }
            __syncwarp();
          }
          bool any = false;
#pragma unroll 8
          for (int c = lane; c < L::kBlock / 16; c += 32) {
            const uint4 w = *reinterpret_cast<const uint4*>(v + c * 16);
            any = any || not_finite(w.x) || not_finite(w.y) || not_finite(w.z) || not_finite(w.w);
          }
          any = __any_sync(0xffffffffu, any);
          if (any) {
            // a lane two columns of 64, keys in falling order: the first one stays
            uint8_t* mine = note + kv % kNotes * D;
#pragma unroll 1
            for (int c = 0; c < D / 64; ++c) {
              int first0 = 64, first1 = 64;
#pragma unroll 1
              for (int r = 63; r >= 0; --r) {
                uint32_t* w = reinterpret_cast<uint32_t*>(v + (r >> 3) * L::kGroup + c * 1024 + (r & 7) * 128 +
                                                          (((lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4);
                const uint32_t x = *w;
                if ((x & 0x7f80u) == 0x7f80u) first0 = r;
                if ((x & 0x7f800000u) == 0x7f800000u) first1 = r;
                if (not_finite(x))
                  *w = x & ((x & 0x7f80u) == 0x7f80u ? 0xffff0000u : ~0u) & ((x & 0x7f800000u) == 0x7f800000u ? 0x0000ffffu : ~0u);
              }
              mine[64 * c + 2 * lane] = static_cast<uint8_t>(first0);
              mine[64 * c + 2 * lane + 1] = static_cast<uint8_t>(first1);
            }
          }
          if (lane == 0) noted[kv % kNotes] = any;
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(kvfull + slot);
        }
        ++kv;
      }
      t = next;
    }
    // every load lands before the CTA may exit (bounded, not abortable)
    if (lane == 0) {
      volatile int no_abort = 0;
      for (uint32_t i = 0; i < L::kKvs && i < kv; ++i)
        mbar_wait(kvfull + (kv - 1 - i) % L::kKvs, ((kv - 1 - i) / L::kKvs) & 1, &no_abort, kWaitLimitNs);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t kQk = idesc_bf16_f32(128, 64, 0), kPv = idesc_bf16_f32(128, D, 1);
      const uint64_t dq = sdesc_sw128(smem_u32(sm_q), 16, 1024), dk = sdesc_sw128(smem_u32(sm_kv), 16, L::kGroup);
      const uint64_t dv = sdesc_sw128(smem_u32(sm_kv) + L::kBlock, 1024, L::kGroup);
      // Scores of tile i and the output of tile j, whichever has what it needs.  Scores go over the P of the tile
      // before the last, whose product was issued before.
      int i = 0, j = 0, cur = -1;
      uint32_t kv = 0, slots = 0, last = 0;  // blocks taken; slots and last tiles of a block of tiles j .. i - 1, low bits first
      bool ok = true;
      int next = n > 0 ? tiles[0].x : 0, after = n > 1 ? tiles[1].x : -1;
      uint64_t since = globaltimer_ns();
#pragma unroll 1
      for (uint32_t idle = 0; j < n;) {
        if (j < i && mbar_test_wait(pfull + (j & 1), (j / 2) & 1) && (j < 2 || mbar_test_wait(ofree + (j & 1), (j / 2 - 1) & 1))) {
          tc_fence_after();
          const uint32_t slot = slots & 0xff;
          const uint64_t w = dv + static_cast<uint64_t>((slot * 2 * L::kBlock) >> 4);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_bf16_ts(tmem + 128 + (j & 1) * D, tmem + (j & 1) * 64 + kk * 8, w + ((kk * 2 * L::kGroup) >> 4), kPv,
                        kk > 0 ? 1u : 0u);
          mma_commit(odone + (j & 1));
          if (last & 1) mma_commit(kvempty + slot);
          slots >>= 8;
          last >>= 1;
          ++j;
          idle = 0;
        }
        const uint32_t q = i % L::kQs, slot = (next != cur ? kv : kv - 1) % L::kKvs;
        if (i < n && i < j + 2 && mbar_test_wait(qfull + q, (i / L::kQs) & 1) &&
            (next == cur || mbar_test_wait(kvfull + slot, (kv / L::kKvs) & 1))) {
          tc_fence_after();
          const uint64_t a = dq + static_cast<uint64_t>((q * L::kQ) >> 4), w = dk + static_cast<uint64_t>((slot * 2 * L::kBlock) >> 4);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t in = (kk & 3) * 32;
            mma_bf16_ss(tmem + (i & 1) * 64, a + (((kk >> 2) * L::kHalf + in) >> 4), w + (((kk >> 2) * 1024 + in) >> 4), kQk,
                        kk > 0 ? 1u : 0u);
          }
          mma_commit(sfull + (i & 1));
          mma_commit(qempty + q);
          if (next != cur) ++kv;
          cur = next;
          slots |= slot << (8 * (i - j));
          last |= (after != cur ? 1u : 0u) << (i - j);
          ++i;
          next = after;
          after = i + 1 < n ? tiles[i + 1].x : -1;
          idle = 0;
        }
        if (++idle == 1) {
          since = globaltimer_ns();
        } else if (idle % 256 == 0) {
          if (*abort_flag) {
            ok = false;
          } else if (globaltimer_ns() - since > kWaitLimitNs) {
            record(21, kDevTimeout);
            *abort_flag = 1;
            ok = false;
          }
          if (!ok) break;
        }
      }
      if (!ok) {
        volatile int no_abort = 0;
        mma_commit(drain);
        mbar_wait(drain, 0, &no_abort, kWaitLimitNs);
      }
    }
  } else if (warp < 4) {
    // Queries: 64 rows a warp, 8 lanes for 128 bytes of a row.  Lane l finds rows l and l + 32 in
    // memory: a tile's description is loaded three tiles ahead, its tokens two.
    const int w2 = warp - 2, sub = lane >> 3, ch = lane & 7;
    const char* q = static_cast<const char*>(p.q) + tok0 * p.Hq * D * 2 + ch * 16;
    const uint32_t tok_step = p.Hq * (D / 8), group_step = G * (D / 8);  // in 16 bytes
    const int e0 = (64 * w2 + lane) / G, e1 = (64 * w2 + lane + 32) / G;
    const uint32_t g0 = (64 * w2 + lane - e0 * G) * (D / 8), g1 = (64 * w2 + lane + 32 - e1 * G) * (D / 8);
    // where a row starts; kNoRow: there is none
    constexpr uint32_t kNoRow = 0xffffffffu;
    struct Found {
      int head, tok0, tok1;  // (KV head, block), tokens
    };
    auto find = [&](const int4& t, int i) {
      const int* at = order + static_cast<long long>(i) * p.tile_tokens;
      return Found{t.x, e0 < t.z ? at[e0] : -1, e1 < t.z ? at[e1] : -1};
    };
    auto place = [&](int head, int tok, uint32_t g) {
      return tok < 0 ? kNoRow : tok * tok_step + static_cast<uint32_t>(head / p.n_blocks) * group_step + g;
    };
    const int4 none = make_int4(0, 0, 0, 0);
    auto tile = [&](int i) { return i < n ? tiles[i] : none; };
    bool ok = true;
    Found now = find(tile(0), 0), next = find(tile(1), 1);
    int4 t = tile(2);
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      const uint32_t slot = i % L::kQs;
      // the tile before the last has landed
      if (i > 1) {
        cp_async_wait<1>();
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(qfull + (i - 2) % L::kQs);
      }
      if (i >= L::kQs) ok = wait_all(qempty + slot, (i / L::kQs - 1) & 1, abort_flag, 31);
      if (!ok) break;
      const uint32_t to = smem_u32(sm_q + slot * L::kQ) + (64 * w2 + sub) * 128;
      const uint32_t at0 = place(now.head, now.tok0, g0), at1 = place(now.head, now.tok1, g1);
      now = next;
      next = find(t, i + 2);
      t = tile(i + 3);
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        // row 64 w2 + 4 k + sub
        const uint32_t at = __shfl_sync(0xffffffffu, k < 8 ? at0 : at1, (4 * k + sub) & 31);
        if (at != kNoRow) {
          const char* from = q + static_cast<size_t>(at) * 16;
          const uint32_t dst = to + k * 512 + ((ch ^ (sub + 4 * (k & 1))) << 4);
#pragma unroll
          for (int c = 0; c < D / 64; ++c) cp_async16(dst + c * L::kHalf, from + c * 128);
        }
      }
      cp_async_commit();
    }
    cp_async_wait<0>();
    fence_proxy_async_smem();
    __syncwarp();
    if (ok && lane == 0) {
      if (n > 1) mbar_arrive(qfull + (n - 2) % L::kQs);
      if (n > 0) mbar_arrive(qfull + (n - 1) % L::kQs);
    }
  } else {
    const int which = (warp - 4) >> 2, row = threadIdx.x - 128 - 128 * which, w4 = warp & 3;
    const int e = row / G;
    const uint32_t lanes = static_cast<uint32_t>(w4) << 21;  // lane 32 w4 of Tensor Memory
    const uint32_t tS = tmem + lanes + which * 64, tO = tmem + lanes + 128 + which * D;
    const float c = p.scale_log2;
    uint8_t* out = smem + L::kOffOut + (warp - 4) * 2 * L::kOut;
    const uint32_t to = smem_u32(out) + lane * 128;
    // tile i and the block of the one before, loaded four tiles ahead, and the row's token of it, two tiles ahead
    const int4 none = make_int4(-1, 0, 0, 0);
    auto tile = [&](int i) { return i < n ? tiles[i] : none; };
    auto token_of = [&](const int4& t, int i) { return e < t.z ? order[static_cast<long long>(i) * p.tile_tokens + e] : 0; };
    int4 t = tile(which), t_next = tile(which + 2);
    int before = which > 0 ? tile(0).x : -1, before_next = tile(which + 1).x, tok = token_of(t, which);
    uint32_t kv = 0;  // blocks up to and with tile i, as the loader numbers them
    int cur = -1;
#pragma unroll 1
    for (int i = which; i < n; i += 2) {
      const int4 t_after = tile(i + 4);
      const int before_after = tile(i + 3).x, tok_next = token_of(t_next, i + 2);
      if (i > 0 && before != cur) ++kv;
      if (i == 0 || t.x != before) ++kv;
      cur = t.x;
      const bool live = e < t.z;
      const int h = t.x / p.n_blocks;
      const int lim = live ? min(64, first_seen + tok - 64 * (t.x - h * p.n_blocks)) : 64;
      const bool masked = __any_sync(0xffffffffu, lim < 64);

      if (!wait_all(sfull + which, (i / 2) & 1, abort_flag, 41)) break;
      tc_fence_after();
      uint32_t u[64];
      tmem_ld32(tS, *reinterpret_cast<uint32_t(*)[32]>(u));
      tmem_ld32(tS + 32, *reinterpret_cast<uint32_t(*)[32]>(u + 32));
      tmem_wait_ld();
      if (masked) {
        const uint32_t least = c < 0.f ? 0x7f800000u : 0xff800000u;
#pragma unroll
        for (int k = 0; k < 64; ++k) u[k] = k < lim ? u[k] : least;
      }
      // the largest s c, from the largest s or, with c < 0, the least
      float m = -INFINITY;
      const uint32_t sign = c < 0.f ? 0x80000000u : 0u;
#pragma unroll
      for (int k = 0; k < 64; k += 2) m = fmax3(m, __uint_as_float(u[k] ^ sign), __uint_as_float(u[k + 1] ^ sign));
      // c = 0: masked scores are told by their place
      const float M = c == 0.f ? 0.f : m * fabsf(c), ref = M == -INFINITY ? 0.f : M;
      float2 a0 = make_float2(0.f, 0.f), a1 = a0;
      const float2 c2 = make_float2(c, c), m2 = make_float2(-ref, -ref);
      uint32_t pk[32];
#pragma unroll
      for (int k = 0; k < 32; ++k) {
        const float2 x = ffma2(make_float2(__uint_as_float(u[2 * k]), __uint_as_float(u[2 * k + 1])), c2, m2);
        float2 y = make_float2(ex2_approx(x.x), ex2_approx(x.y));
        if (masked) {
          if (2 * k >= lim) y.x = 0.f;
          if (2 * k + 1 >= lim) y.y = 0.f;
        }
        if (k & 1)
          a1 = fadd2(a1, y);
        else
          a0 = fadd2(a0, y);
        pk[k] = pack_bf16x2(y.x, y.y);
      }
      tmem_st32(tS, pk);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(pfull + which);
      const float l = (a0.x + a0.y) + (a1.x + a1.y), inv = l == 0.f ? 0.f : 1.f / l;

      if (!wait_all(odone + which, (i / 2) & 1, abort_flag, 42)) break;
      tc_fence_after();
      const bool notes = noted[(kv - 1) % kNotes] != 0;
      // rows of 128 bytes, 16 at a time exchanged by the row: the map's order, and no two lanes on a bank
#pragma unroll
      for (int s = 0; s < D / 32; ++s) {
        if (lane == 0) bulk_wait_read<1>();  // this half of the buffer is free
        __syncwarp();
        tmem_ld32(tO + 32 * s, *reinterpret_cast<uint32_t(*)[32]>(u));
        tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < 32; ++k) u[k] = __float_as_uint(__uint_as_float(u[k]) * inv);
        if (notes) {
          const uint8_t* at = note + (kv - 1) % kNotes * D + 32 * s;
#pragma unroll
          for (int k = 0; k < 32; ++k)
            if (at[k] < lim) u[k] = 0x7fc00000u;
        }
#pragma unroll
        for (int k = 0; k < 8; ++k)
          st_shared_v4(to + (s & 1) * L::kOut + ((k ^ (lane & 7)) << 4), u[4 * k], u[4 * k + 1], u[4 * k + 2], u[4 * k + 3]);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          if (32 * w4 < t.z * G) tma_store_2d(&tm_o, out + (s & 1) * L::kOut, 32 * s, 32 * (t.y + w4));
          bulk_commit();
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(ofree + which);
      if (live) p.lse_part[32ll * t.y + row] = l == 0.f ? -INFINITY : M + __log2f(l);
      tok = tok_next;
      t = t_next;
      t_next = t_after;
      before = before_next;
      before_next = before_after;
    }
    if (lane == 0) bulk_wait<0>();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, L::kTmem);
  }
}

// A chunk's rows joined from their entries' pieces.
template <int D>
__global__ void __launch_bounds__(32 * kJoinWarps) join_entries_kernel(const __grid_constant__ ByBlockParams p, int group) {
  grid_depends();
  const int G = p.Hq / p.Hkv, b = group / p.chunks, i0 = (group - b * p.chunks) * p.chunk_tokens;
  const int row = blockIdx.x * kJoinWarps + (threadIdx.x >> 5);
  const int i = row / p.Hq, hq = row - i * p.Hq, h = hq / G;
  if (i >= min(p.chunk_tokens, p.Nq - i0)) return;
  const int tok = b * p.Nq + i0 + i, seen = seen_by(p, b, i0 + i);
  const int* list = p.blocks + (static_cast<long long>(tok) * p.Hkv + h) * p.n_sel;
  const int* rank = p.rank + (static_cast<long long>(tok) * p.Hkv + h) * p.n_sel;
  const int2* starts = p.starts + (static_cast<long long>(group) * p.Hkv + h) * p.n_blocks;
  Join s = {-INFINITY, 0.f};
  float acc[D / 32];
#pragma unroll
  for (int x = 0; x < D / 32; ++x) acc[x] = 0.f;
  join<D>(p, p.n_sel,
          [&](int x) {
            const int blk = list[x];
            if (blk < 0 || blk >= p.n_blocks || blk * 64 >= seen) return -1ll;
            const int r = rank[x], t = static_cast<int>(p.tile_len.div(static_cast<uint32_t>(r)));
            return 32ll * starts[blk].y + 128 * t + (r - t * p.tile_tokens) * G + hq - h * G;
          },
          s, acc);
  write_row<D>(p, tok, hq, s, acc);
}

template <int D>
cudaError_t launch_d(const ByBlockParams& p, const CUtensorMap& tm_k, const CUtensorMap& tm_v, const CUtensorMap& tm_o,
                     cudaStream_t stream) {
  using L = Layout<D>;
  int dev = 0, n_sm = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, dev);
  auto kern = by_block_kernel<D>;
  if (e == cudaSuccess) e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kAlloc);
  const int groups = p.B * p.chunks;
  if (e == cudaSuccess)
    e = cudaMemsetAsync(p.counts, 0, static_cast<size_t>(groups) * p.Hkv * p.n_blocks * sizeof(int), stream);
  if (e != cudaSuccess) return e;
  const long long lists = static_cast<long long>(p.B) * p.Nq * p.Hkv;
  const dim3 sort(static_cast<unsigned>((lists + kSortWarps - 1) / kSortWarps));
  count_kernel<<<sort, 32 * kSortWarps, 0, stream>>>(p);
  e = cudaGetLastError();
  if (e == cudaSuccess) e = launch_dependent(plan_kernel, dim3(groups * p.Hkv), kPlanThreads, 0, stream, p);
  if (e == cudaSuccess) e = launch_dependent(place_kernel, sort, 32 * kSortWarps, 0, stream, p);
  const unsigned rows = static_cast<unsigned>((static_cast<long long>(p.chunk_tokens) * p.Hq + kJoinWarps - 1) / kJoinWarps);
  for (int g = 0; g < groups && e == cudaSuccess; ++g) {
    e = launch_dependent(kern, dim3(n_sm), kThreads, L::kAlloc, stream, tm_k, tm_v, tm_o, p, g);
    if (e == cudaSuccess) e = launch_dependent(join_entries_kernel<D>, dim3(rows), 32 * kJoinWarps, 0, stream, p, g);
  }
  return e;
}

}  // namespace

ByBlockSizes by_block_sizes(int B, int Nq, int Hq, int Hkv, int d, int n_sel, long long n_blocks) {
  ByBlockSizes z = {};
  const int G = Hq / Hkv;
  const long long lists = static_cast<long long>(B) * Nq * Hkv;
  if (G > kByBlockHeads || lists > (1LL << 30) / n_sel) return z;
  const int T = 128 / G;
  const long long blocks = Hkv * n_blocks;
  long long ct = kByBlockBytes / (static_cast<long long>(Hq) * n_sel * d * 4);
  if (ct > Nq) ct = Nq;
  if (ct < 1) return z;
  z.chunks = static_cast<int>((Nq + ct - 1) / ct);
  z.chunk_tokens = (Nq + z.chunks - 1) / z.chunks;
  const long long entries = static_cast<long long>(z.chunk_tokens) * Hkv * n_sel;
  if (entries < kByBlockEntries || entries < kByBlockShare * blocks) return ByBlockSizes{};
  z.tile_tokens = T;
  z.tile_cap = entries / T + (entries < blocks ? entries : blocks);
  // full tiles take 128 rows, a block's last one up to 31 more than its entries have
  z.rows = (entries / T * 128 + (entries % T) * G + 31 * (entries < blocks ? entries : blocks) + 31) / 32 * 32;
  z.groups = static_cast<long long>(B) * z.chunks;
  z.entries = lists * n_sel;
  return z;
}

cudaError_t launch_by_block(const ByBlockParams& p, const CUtensorMap& tm_k, const CUtensorMap& tm_v, const CUtensorMap& tm_o,
                            cudaStream_t stream) {
  return p.d == 64 ? launch_d<64>(p, tm_k, tm_v, tm_o, stream) : launch_d<128>(p, tm_k, tm_v, tm_o, stream);
}

cudaError_t status_word_by_block(uint32_t** at) { return cudaGetSymbolAddress(reinterpret_cast<void**>(at), g_rows_status); }

}  // namespace attn

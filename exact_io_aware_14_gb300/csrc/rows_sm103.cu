// Attention of query rows over a paged bf16 cache, for sm_103a: over whole
// sequences whose first keys the batch shares (attn_fwd_splitkv_paged_shared),
// or over listed 64-key blocks (attn_fwd_blocks_paged); here where more than 32
// rows read the same keys (few_rows_sm103.cu takes fewer).
//
// A row is a query token and one of the heads that read a KV head.  S = Q K^T
// and O += P V run on tcgen05 with 128 rows and 128 keys a tile.  The rows of a
// tile are all that read the same keys: for the shared prefix the tokens of the
// whole batch with the heads of a group, for a sequence's own keys its new
// tokens with theirs, for listed blocks one token's heads.  A product of 128
// rows and keys of d = 128 takes 512 cycles whatever part of the rows is there.
//
// Work is cut into equal runs of tiles, whatever the lengths.  A CTA has two
// slots, each with a tile of rows, its scores, its accumulator and a
// warpgroup for its softmax.
//   Pair work (a prefix read by more rows than one tile): the slots hold two
//     tiles of rows and share every K/V tile; each CTA takes an equal run of
//     (KV head, pair, key tile).  Bound by the issue of products: 64 sequences
//     with 32 heads on a prefix of 131072 keys, 8 KV heads of d = 128, take
//     131 us in all, 137 GFLOP at 1.05 PFLOP/s (2350 of a step's 3500 cycles
//     the tensor core has a product; the rest goes into waits for P).
//   Lane work (all else): each slot is a lane of its own with its own K/V
//     tiles, and each lane takes an equal run of (unit, key tile), a unit being
//     the rows and keys named above.
// What a lane computes of a unit is a piece; pieces of a row (normalised O and
// log-sum-exp, fp32) go to the workspace, and a second kernel joins them in
// order.  A piece of listed blocks that is a whole unit is written as result.
// Piece numbers need no counters: along the runs either the lane or the unit
// goes up by one, so lane + unit is a number of its own for each piece.
//
// P is rounded to bf16, the tensor core's operand; its sum takes it before.
//
// Warps: 0 producer (work, pages, TMA loads into one ring in the order of use),
// 1 MMA issuer, 2 clears value rows that hold anything, 4-7 and 8-11 softmax
// and results of slots 0 and 1.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "launch.h"
#include "ptx.cuh"
#include "rows_join.cuh"
#include "rows_plan.cuh"
#include "rows_softmax.cuh"

namespace attn {
namespace {

constexpr int kThreads = 384;
constexpr uint32_t kTmemCols = 512;

// What a slot computes next, as the producer tells the other warps.
struct Piece {
  int n;      // key tiles; -1: no more work
  int share;  // 0 own K/V tiles; 1 those of both slots; 2 the same, slot 1 without rows
  int h;      // KV head
  int tok0, ntok;  // first token, tokens
  int key0, keys;  // ranges: position of the first tile's first key, keys from there on
  int dst;    // piece number, -1: the result itself
  int part;   // keys seen of the blocks marked in some[] (lists)
  uint32_t full[kMaskWords], some[kMaskWords];  // lists: blocks seen whole, seen in part
};
template <int D>
struct Layout {
  static constexpr int kSlots = D == 64 ? 10 : 5;
  static constexpr int kHalf = 128 * 128;  // one 64-column block of a 128-row tile
  static constexpr int kTile = 128 * D * 2;
  // K and V tiles: groups of 8 keys, each with its D / 64 blocks of 8 rows of
  // 128 B, so that one box holds a 64-key block and both halves follow on
  static constexpr int kGroup = D / 64 * 1024;
  static constexpr int kOffRing = 2 * kTile;
  static constexpr int kOffPiece = kOffRing + kSlots * kTile;
  static constexpr int kOffBar = kOffPiece + 4 * static_cast<int>(sizeof(Piece));
  static constexpr int kNumBars = 2 * kSlots + 6 * 2 + 2 * 4 + 3 * 4 + 1;
  static constexpr int kOffFix = kOffBar + 8 * kNumBars;
  static constexpr int kOffPlan = (kOffFix + 4 * static_cast<int>(sizeof(Fix)) + 15) & ~15;
  static constexpr int kOffScan = kOffPlan + static_cast<int>(sizeof(Plan));
  static constexpr int kOffMisc = kOffScan + 12 * 8 + 2 * 12 * 4;
  static constexpr int kBytes = kOffMisc + 16;
  static constexpr int kAlloc = kBytes + 1024;  // slack to align the base to 1024 B
};
static_assert(Layout<128>::kAlloc <= 232448 && Layout<64>::kAlloc <= 232448, "shared memory of a CTA");

// The lane of a slot: with few runs the CTAs have one each.
__device__ __forceinline__ int lane_of(int slot) { return slot * static_cast<int>(gridDim.x) + static_cast<int>(blockIdx.x); }

// Shared memory of a CTA.
template <int D>
struct Smem {
  uint8_t *q, *ring;
  Piece* pieces;         // [slot][2]
  uint64_t* full;        // [kSlots] ring slot holds its tile
  uint64_t* empty;       // [kSlots] ring slot read
  uint64_t* sfull;       // [2] scores complete
  uint64_t* pfull;       // [2] P written (4 warps)
  uint64_t* odone;       // [2] a piece's last P V complete
  uint64_t* ofree;       // [2] a piece's O read (4 warps)
  uint64_t* qfull;       // [2] rows loaded
  uint64_t* qfree;       // [2] a piece's last Q K^T complete
  uint64_t* pieced;      // [slot][2] piece told
  uint64_t* unpieced;    // [slot][2] piece done with (MMA thread, 4 warps)
  uint64_t* fixset;      // [4] clearing asked for
  uint64_t* fixdone;     // [4] done
  uint64_t* raw;         // [4] value tile to be cleared landed
  uint64_t* drain;       // after an abort: the MMAs issued so far completed
  Fix* fixes;
  Plan* plan;
  volatile int* abort_flag;
  uint32_t* tmem_slot;
  __device__ __forceinline__ explicit Smem(uint8_t* base) {
    using L = Layout<D>;
    q = base;
    ring = base + L::kOffRing;
    pieces = reinterpret_cast<Piece*>(base + L::kOffPiece);
    full = reinterpret_cast<uint64_t*>(base + L::kOffBar);
    empty = full + L::kSlots;
    sfull = empty + L::kSlots;
    pfull = sfull + 2;
    odone = pfull + 2;
    ofree = odone + 2;
    qfull = ofree + 2;
    qfree = qfull + 2;
    pieced = qfree + 2;
    unpieced = pieced + 4;
    fixset = unpieced + 4;
    fixdone = fixset + 4;
    raw = fixdone + 4;
    drain = raw + 4;
    fixes = reinterpret_cast<Fix*>(base + L::kOffFix);
    plan = reinterpret_cast<Plan*>(base + L::kOffPlan);
    tmem_slot = reinterpret_cast<uint32_t*>(base + L::kOffMisc);
    abort_flag = reinterpret_cast<volatile int*>(base + L::kOffMisc + 4);
  }
};

// ---------------------------------------------------------------------------
// Producer: one warp, whose lanes look up 32 blocks of a piece at a time; lane 0
// waits and issues.  What belongs to a slot is in a struct; the two take turns in
// the same registers and the same code (exchanged after each step), so that no
// state lies in local memory and the code is there once.
struct ProducerSlot {
  // the lane's run
  long long left;        // tiles left (lists: of the cut units)
  long long unit;        // lists: next whole unit
  int b, h, rt, t;       // ranges: where it stands
  // the piece being loaded
  int n, j, head;
  int key0, end, row;    // ranges: first key, end of the keys; table row
  const int* list;       // lists: entries of the piece, `count` of them
  int count, seen;       // seen: keys before the token's own end
  int blk;               // first group of 8 keys of this lane's block of the 32 looked up
  uint32_t seen_bits, full_bits;
  int part;
  Tile last;             // the tile whose V comes next
  uint32_t told, rows_n;  // pieces told, rows loaded
  int slot;
  bool fin, pend;
};
template <typename T>
__device__ __forceinline__ void exchange(T& a, T& b) {
  const T t = a;
  a = b;
  b = t;
}

template <int D, bool kList>
struct Producer {
  using L = Layout<D>;
  const RowsParams& p;
  const CUtensorMap *tm_q, *tm_qs, *tm_k, *tm_v;
  const Smem<D>& sm;
  const int lane;
  RingAt<L::kSlots> at;
  uint32_t fix_n = 0;
  bool ok = true;  // lane 0's view until `agree`

  __device__ __forceinline__ Producer(const RowsParams& p_, const CUtensorMap* q, const CUtensorMap* qs, const CUtensorMap* k,
                                      const CUtensorMap* v, const Smem<D>& sm_, int lane_)
      : p(p_), tm_q(q), tm_qs(qs), tm_k(k), tm_v(v), sm(sm_), lane(lane_) {}

  __device__ __forceinline__ void wait(uint64_t* bar, uint32_t parity, uint32_t site) {
    if (ok) ok = wait_one(bar, parity & 1, sm.abort_flag, site);
  }
  __device__ __forceinline__ bool agree() {
    ok = __shfl_sync(0xffffffffu, static_cast<int>(ok), 0) != 0;
    return ok;
  }

  // blocks 32 i .. 32 i + 31 of the piece
  __device__ __forceinline__ void look_up(ProducerSlot& s, int i) {
    int v = 0, blk;
    if (kList) {
      const int e = 32 * i + lane;
      blk = e < s.count ? s.list[e] : -1;
      if (blk >= 0) {
        if (blk >= p.max_blocks * (p.page_size / 64))
          record(3, kDevBadPage);
        else
          v = min(64, s.seen - blk * 64);
      }
    } else {
      const int key = s.key0 + 64 * (32 * i + lane);
      v = min(64, s.end - key);
      blk = key >> 6;
    }
    s.blk = 0;
    if (v > 0) s.blk = pool_group(p, s.row, blk);
    s.seen_bits = __ballot_sync(0xffffffffu, v > 0);
    s.full_bits = __ballot_sync(0xffffffffu, v == 64);
    const uint32_t some = s.seen_bits & ~s.full_bits;
    s.part = some ? __shfl_sync(0xffffffffu, v, __ffs(some) - 1) : 0;  // the same for all of them
  }
  __device__ __forceinline__ Tile tile(const ProducerSlot& s, int j) {
    const int e = 2 * (j & 15);
    Tile t;
    t.g0 = __shfl_sync(0xffffffffu, s.blk, e);
    t.g1 = __shfl_sync(0xffffffffu, s.blk, e + 1);
    t.flags = (s.seen_bits >> e & 3u) | (s.full_bits >> e & 3u) << 2;
    t.part = s.part;
    return t;
  }
  // a K or V tile into the next ring slot
  __device__ __forceinline__ void load(const Tile& t, int h, bool is_v) {
    if (lane != 0) return;
    if (at.turn > 0) wait(sm.empty + at.slot, at.turn - 1, 11);
    if (!ok) return;
    uint8_t* dst = sm.ring + at.slot * L::kTile;
    const CUtensorMap* tm = is_v ? tm_v : tm_k;
    if (t.flags == 15u) {
      uint64_t* done = sm.full + at.slot;
      mbar_arrive_expect_tx(done, L::kTile);
      tma_load_5d(dst, tm, done, 0, 0, 0, t.g0, h);
      tma_load_5d(dst + L::kTile / 2, tm, done, 0, 0, 0, t.g1, h);
    } else {
      const bool s0 = t.flags & 1u, s1 = t.flags & 2u;
      const uint32_t fi = fix_n & 3;
      uint64_t* done = is_v ? sm.raw + fi : sm.full + at.slot;
      if (is_v) {
        if (fix_n >= 4) wait(sm.fixdone + fi, fix_n / 4 - 1, 12);
        if (!ok) return;
        sm.fixes[fi].slot = static_cast<int>(at.slot);
        sm.fixes[fi].v0 = t.flags & 4u ? 64 : (s0 ? t.part : 0);
        sm.fixes[fi].v1 = t.flags & 8u ? 64 : (s1 ? t.part : 0);
      }
      if (s0 || s1)
        mbar_arrive_expect_tx(done, s0 && s1 ? L::kTile : L::kTile / 2);
      else
        mbar_arrive(done);
      if (s0) tma_load_5d(dst, tm, done, 0, 0, 0, t.g0, h);
      if (s1) tma_load_5d(dst + L::kTile / 2, tm, done, 0, 0, 0, t.g1, h);
      if (is_v) {
        mbar_arrive(sm.fixset + fi);
        ++fix_n;
      }
    }
    at.next();
  }
  // the place of the slot's next piece, once it is free
  __device__ __forceinline__ Piece& place(const ProducerSlot& s) {
    if (lane == 0 && s.told >= 2) wait(sm.unpieced + s.slot * 2 + (s.told & 1), s.told / 2 - 1, 13);
    return sm.pieces[s.slot * 2 + (s.told & 1)];
  }
  __device__ __forceinline__ void tell(ProducerSlot& s, Piece& d, int n, int share, int h, int tok0, int ntok, int key0, int keys,
                                       int dst) {
    if (lane == 0 && ok) {
      d.n = n;
      d.share = share;
      d.h = h;
      d.tok0 = tok0;
      d.ntok = ntok;
      d.key0 = key0;
      d.keys = keys;
      d.dst = dst;
      mbar_arrive(sm.pieced + s.slot * 2 + (s.told & 1));
    }
    ++s.told;
  }
  // the rows of a piece
  __device__ __forceinline__ void load_rows(ProducerSlot& s, bool pair, int h, int tok0) {
    if (lane != 0) return;
    if (s.rows_n > 0) wait(sm.qfree + s.slot, s.rows_n - 1, 14);
    if (!ok) return;
    const int tokens = pair ? p.tile_tokens : p.unit_tokens;
    mbar_arrive_expect_tx(sm.qfull + s.slot, static_cast<uint32_t>(tokens * (p.Hq / p.Hkv) * D * 2));
#pragma unroll
    for (int c = 0; c < D / 64; ++c)
      tma_load_4d(sm.q + s.slot * L::kTile + c * L::kHalf, pair ? tm_q : tm_qs, sm.qfull + s.slot, c * 64, 0, h, tok0);
    ++s.rows_n;
  }

  // Pair work: pieces of the CTA's run, each to its end.
  __device__ __forceinline__ void pair_work(ProducerSlot& a, ProducerSlot& b) {
    const int end = sm.plan->prefix_end, nt = tiles_of(end), grid = gridDim.x, tokens = p.B * p.Nq;
    long long x = run_start(sm.plan->pair_total, grid, blockIdx.x);
    const long long x1 = run_start(sm.plan->pair_total, grid, blockIdx.x + 1);
    while (x < x1 && agree()) {
      const int unit = static_cast<int>(x / nt), t = static_cast<int>(x - static_cast<long long>(unit) * nt);
      const int n = static_cast<int>(min(static_cast<long long>(nt - t), x1 - x));
      const int h = unit / p.pairs, pair = unit - h * p.pairs;
      const int tok0 = 2 * pair * p.tile_tokens, tok1 = tok0 + p.tile_tokens;
      const int share = tok1 < tokens ? 1 : 2, dst = static_cast<int>(blockIdx.x) + unit;
      a.key0 = 128 * t;
      a.end = end;
      a.row = 0;
      Piece& d0 = place(a);
      tell(a, d0, n, share, h, tok0, min(p.tile_tokens, tokens - tok0), a.key0, end - a.key0, dst);
      Piece& d1 = place(b);
      tell(b, d1, n, share, h, tok1, max(0, min(p.tile_tokens, tokens - tok1)), a.key0, end - a.key0, dst);
      load_rows(a, true, h, tok0);
      if (share == 1) load_rows(b, true, h, tok1);
      for (int j = 0; j <= n; ++j) {
        if (j > 0) load(a.last, h, true);
        if (j == n) break;
        if ((j & 15) == 0) look_up(a, j >> 4);
        a.last = tile(a, j);
        load(a.last, h, false);
      }
      x += n;
    }
  }

  // Next piece of a slot: told, its rows on their way; n = 0 where there is none or nothing to compute.
  __device__ __forceinline__ void next_piece(ProducerSlot& s) {
    const int l = lane_of(s.slot), lanes = 2 * gridDim.x;
    Piece& d = place(s);
    int tok0, ntok, dst;
    s.j = 0;
    if (kList) {
      const int units = p.B * p.Nq * p.Hkv, unit_tiles = (p.n_sel + 1) >> 1;
      const int whole = units / lanes * lanes;
      const long long cut = static_cast<long long>(units - whole) * unit_tiles;
      long long u;
      int t0 = 0, nt = unit_tiles;
      dst = -1;
      if (s.unit < whole) {
        u = s.unit;
        s.unit += lanes;
      } else if (s.left > 0) {
        const long long first = run_start(cut, lanes, l), x = run_start(cut, lanes, l + 1) - s.left;
        const int cu = static_cast<int>(x / unit_tiles);
        u = whole + cu;
        t0 = static_cast<int>(x - static_cast<long long>(cu) * unit_tiles);
        nt = static_cast<int>(min(static_cast<long long>(unit_tiles - t0), s.left));
        if (nt < unit_tiles) dst = 2 * l + (x > first ? 1 : 0);
        s.left -= nt;
      } else {
        s.fin = true;
        s.n = 0;
        tell(s, d, -1, 0, 0, 0, 0, 0, 0, 0);
        return;
      }
      // units by sequence, head, token: neighbours read the same head's keys
      const int per = p.Hkv * p.Nq;
      const int b = static_cast<int>(u / per), r = static_cast<int>(u - static_cast<long long>(b) * per);
      s.head = r / p.Nq;
      const int i = r - s.head * p.Nq;
      tok0 = b * p.Nq + i;
      ntok = 1;
      const int len = clamped_len(p, b);
      if (lane == 0 && s.head == 0 && i == 0 && t0 == 0 && len != p.seqlens[b]) record(1, kDevBadSeqlen);
      s.row = b;
      s.seen = max(0, len - p.Nq + i + 1);
      s.list = p.blocks + (static_cast<long long>(tok0) * p.Hkv + s.head) * p.n_sel + 2 * t0;
      s.count = min(p.n_sel - 2 * t0, 2 * nt);
      s.key0 = s.end = 0;
      // which of them are seen; the last one that is ends the piece
      int last = -1;
      for (int w = (s.count - 1) >> 5; w >= 0; --w) {  // ends with the first 32 looked up
        look_up(s, w);
        if (lane == 0 && ok) {
          d.full[w] = s.full_bits;
          d.some[w] = s.seen_bits & ~s.full_bits;
          if (d.some[w]) d.part = s.part;
        }
        if (last < 0 && s.seen_bits) last = 32 * w + 31 - __clz(s.seen_bits);
      }
      s.n = (last + 2) >> 1;
    } else {
      if (s.left == 0) {
        s.fin = true;
        s.n = 0;
        tell(s, d, -1, 0, 0, 0, 0, 0, 0, 0);
        return;
      }
      int len = s.b < 0 ? 0 : clamped_len(p, s.b);
      while (s.b >= 0 && len <= p.shared_len) len = clamped_len(p, ++s.b);  // a sequence with keys of its own is ahead
      int nt, rts, unit;
      s.head = s.h;
      if (s.b < 0) {
        s.end = sm.plan->prefix_end;
        s.key0 = 128 * s.t;
        s.row = 0;
        nt = tiles_of(s.end);
        rts = 1;
        unit = s.h;
        tok0 = 0;
        ntok = p.B * p.Nq;
      } else {
        s.end = len;
        s.key0 = p.shared_len + 128 * s.t;
        s.row = s.b;
        nt = tiles_of(len - p.shared_len);
        rts = p.own_rt;
        unit = (s.b * p.Hkv + s.h) * rts + s.rt + (p.pairs ? 0 : p.Hkv);
        tok0 = s.b * p.Nq + s.rt * p.own_tokens;
        ntok = min(p.own_tokens, p.Nq - s.rt * p.own_tokens);
      }
      dst = l + unit;
      s.n = static_cast<int>(min(static_cast<long long>(nt - s.t), s.left));
      s.left -= s.n;
      s.t += s.n;
      if (s.t == nt) {
        s.t = 0;
        if (++s.rt == rts) {
          s.rt = 0;
          if (++s.h == p.Hkv) {
            s.h = 0;
            ++s.b;
          }
        }
      }
    }
    tell(s, d, s.n, 0, s.head, tok0, ntok, s.key0, s.end - s.key0, dst);
    if (s.n == 0) return;
    load_rows(s, false, s.head, tok0);
    if (!kList) look_up(s, 0);
  }

  __device__ __forceinline__ void start_lane(ProducerSlot& s) {
    const int l = lane_of(s.slot), lanes = 2 * gridDim.x;
    s.n = s.j = 0;
    if (kList) {
      const int units = p.B * p.Nq * p.Hkv;
      const long long cut = static_cast<long long>(units - units / lanes * lanes) * ((p.n_sel + 1) >> 1);
      s.unit = l;
      s.left = run_start(cut, lanes, l + 1) - run_start(cut, lanes, l);
    } else {
      const long long total = sm.plan->total;
      s.left = p.only_pairs ? 0 : run_start(total, lanes, l + 1) - run_start(total, lanes, l);
      if (s.left > 0) {
        s.b = sm.plan->lane_b[s.slot];
        const int nt = s.b < 0 ? tiles_of(sm.plan->prefix_end) : own_tiles(p, s.b), rts = s.b < 0 ? 1 : p.own_rt;
        const long long x = sm.plan->lane_at[s.slot];
        const int u = static_cast<int>(x / nt);
        s.h = u / rts;
        s.rt = u - s.h * rts;
        s.t = static_cast<int>(x - static_cast<long long>(u) * nt);
      }
    }
  }

  __device__ __forceinline__ void lane_step(ProducerSlot& s) {
    if (s.pend) load(s.last, s.head, true);
    s.pend = false;
    while (!s.fin && s.j == s.n && agree()) next_piece(s);
    if (s.fin) return;  // the lanes part nowhere else: what lane 0 alone knows of a failure only keeps it from issuing
    if (s.j > 0 && (s.j & 15) == 0) look_up(s, s.j >> 4);
    s.last = tile(s, s.j);
    load(s.last, s.head, false);
    ++s.j;
    s.pend = true;
  }

  __device__ __forceinline__ void run() {
    ProducerSlot a, b;
    a.told = b.told = a.rows_n = b.rows_n = 0;
    a.fin = b.fin = a.pend = b.pend = false;
    a.slot = 0;
    b.slot = 1;
    if (!kList && sm.plan->pair_total > 0) pair_work(a, b);
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
      start_lane(a);
      exchange(a, b);
    }
#pragma unroll 1
    while (agree() && !(a.fin && b.fin && !a.pend && !b.pend)) {
      lane_step(a);
      exchange(a, b);
    }
    if (a.slot) exchange(a, b);
    if (lane != 0) return;
    if (ok) {
      // no more to clear
      const uint32_t fi = fix_n & 3;
      if (fix_n >= 4) wait(sm.fixdone + fi, fix_n / 4 - 1, 12);
      if (ok) {
        sm.fixes[fi].slot = -1;
        mbar_arrive(sm.fixset + fi);
      }
    }
    // every load lands before the CTA may exit, whatever became of the others (bounded, not abortable)
    volatile int no_abort = 0;
    auto drain = [&](uint64_t* bar, uint32_t parity) { mbar_wait(bar, parity & 1, &no_abort, kWaitLimitNs); };
    if (a.rows_n) drain(sm.qfull + 0, a.rows_n - 1);
    if (b.rows_n) drain(sm.qfull + 1, b.rows_n - 1);
#pragma unroll 1
    for (uint32_t i = 0; i < 4 && i < fix_n; ++i) drain(sm.raw + i, (fix_n - 1 - i) / 4);
#pragma unroll 1
    for (uint32_t i = 0; i < L::kSlots; ++i) {
      const uint32_t turns = at.turn + (i < at.slot ? 1 : 0);
      if (turns > 0) drain(sm.full + i, turns - 1);
    }
  }
};

// ---------------------------------------------------------------------------
// MMA issuer: one thread.
struct MmaSlot {
  int n, j;
  uint32_t seen, done, tiles;  // pieces looked at, with products; P tiles consumed
  uint32_t rows_n;             // rows used
  bool fin, pend;
};

template <int D>
struct Issuer {
  using L = Layout<D>;
  static constexpr uint32_t kIdescQk = idesc_bf16_f32(128, 128, 0), kIdescPv = idesc_bf16_f32(128, D, 1);
  const Smem<D>& sm;
  const uint32_t tmem;
  uint64_t dQ, dK, dV;
  RingAt<L::kSlots> at;
  bool ok = true;

  __device__ __forceinline__ Issuer(const Smem<D>& sm_, uint32_t tmem_) : sm(sm_), tmem(tmem_) {
    dQ = sdesc_sw128(smem_u32(sm.q), 16, 1024);
    dK = sdesc_sw128(smem_u32(sm.ring), 16, L::kGroup);
    dV = sdesc_sw128(smem_u32(sm.ring), 1024, L::kGroup);
  }
  __device__ __forceinline__ void wait(uint64_t* bar, uint32_t parity, uint32_t site) {
    if (ok) ok = wait_one(bar, parity & 1, sm.abort_flag, site);
  }
  // O_S (+)= P_S V, S_S = Q_S K^T with the tile in ring slot `slot`
  template <int S>
  __device__ __forceinline__ void pv(uint32_t slot, bool first) {
    const uint64_t dv = dV + static_cast<uint64_t>((slot * L::kTile) >> 4);
#pragma unroll
    for (int kk = 0; kk < 8; ++kk)
      mma_bf16_ts(tmem + 256 + S * 128, tmem + S * 128 + kk * 8, dv + ((kk * 2 * L::kGroup) >> 4), kIdescPv,
                  (!first || kk > 0) ? 1u : 0u);
  }
  template <int S>
  __device__ __forceinline__ void qk(uint32_t slot) {
    const uint64_t da = dQ + static_cast<uint64_t>((S * L::kTile) >> 4);
    const uint64_t db = dK + static_cast<uint64_t>((slot * L::kTile) >> 4);
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      const uint32_t in = (kk & 3) * 32;
      mma_bf16_ss(tmem + S * 128, da + (((kk >> 2) * L::kHalf + in) >> 4), db + (((kk >> 2) * 1024 + in) >> 4), kIdescQk,
                  kk > 0 ? 1u : 0u);
    }
    mma_commit(sm.sfull + S);
  }
  // Next piece of a slot; false where there is none to come.
  template <int S>
  __device__ __forceinline__ void take(MmaSlot& s, int* share) {
    const uint32_t i = S * 2 + (s.seen & 1);
    wait(sm.pieced + i, s.seen / 2, 24);
    if (!ok) return;
    const volatile Piece& d = sm.pieces[i];
    s.n = d.n;
    *share = d.share;
    mbar_arrive(sm.unpieced + i);
    ++s.seen;
    s.j = 0;
    s.fin = s.n < 0;
    if (s.fin) s.n = 0;
  }

  // One piece of pair work (told to both slots), tiles in the ring as K_0, then
  // V_{j-1}, K_j, and V_{n-1}.  Every instruction of this thread between two
  // products leaves the tensor core idle, so a step probes the barriers that come
  // next right behind a batch, while it still runs, and waits only for those that
  // were not complete.
  __device__ __forceinline__ bool await(uint64_t* bar, uint32_t parity, uint32_t site) {
    return wait_one(bar, parity & 1, sm.abort_flag, site);
  }
  __device__ __forceinline__ bool pair_piece(MmaSlot& a, MmaSlot& b) {
    const int n = a.n;
    if (!await(sm.qfull + 0, a.rows_n++, 26) || !await(sm.qfull + 1, b.rows_n++, 26) || !await(sm.full + at.slot, at.turn, 25))
      return false;
    tc_fence_after();
    qk<0>(at.slot);
    qk<1>(at.slot);
    mma_commit(sm.empty + at.slot);
    at.next();
    if (a.done > 0 && !await(sm.ofree + 0, a.done - 1, 23)) return false;
    if (b.done > 0 && !await(sm.ofree + 1, b.done - 1, 23)) return false;
    uint32_t p0 = a.tiles & 1, p1 = b.tiles & 1;
    bool v_ready = false, p0_ready = false;
#pragma unroll 1
    for (int j = 1; j < n; ++j) {
      const uint32_t vs = at.slot, vt = at.turn & 1;
      at.next();
      const uint32_t ks = at.slot, kt = at.turn & 1;
      at.next();
      if (!v_ready && !await(sm.full + vs, vt, 21)) return false;
      if (!p0_ready && !await(sm.pfull + 0, p0, 22)) return false;
      tc_fence_after();
      pv<0>(vs, j == 1);
      const bool k_ready = mbar_test_wait(sm.full + ks, kt);
      if (!k_ready && !await(sm.full + ks, kt, 25)) return false;
      qk<0>(ks);
      const bool p1_ready = mbar_test_wait(sm.pfull + 1, p1);
      if (!p1_ready && !await(sm.pfull + 1, p1, 22)) return false;
      tc_fence_after();
      pv<1>(vs, j == 1);
      qk<1>(ks);
      mma_commit(sm.empty + vs);
      mma_commit(sm.empty + ks);
      p0 ^= 1;
      p1 ^= 1;
      v_ready = mbar_test_wait(sm.full + at.slot, at.turn & 1);
      p0_ready = mbar_test_wait(sm.pfull + 0, p0);
    }
    mma_commit(sm.qfree + 0);
    mma_commit(sm.qfree + 1);
    if (!await(sm.full + at.slot, at.turn, 21) || !await(sm.pfull + 0, p0, 22)) return false;
    tc_fence_after();
    pv<0>(at.slot, n == 1);
    mma_commit(sm.odone + 0);
    if (!await(sm.pfull + 1, p1, 22)) return false;
    tc_fence_after();
    pv<1>(at.slot, n == 1);
    mma_commit(sm.odone + 1);
    mma_commit(sm.empty + at.slot);
    at.next();
    a.tiles += n;
    b.tiles += n;
    ++a.done;
    ++b.done;
    return true;
  }
  // The same where slot 1 has no rows.
  __device__ __forceinline__ bool single_piece(MmaSlot& a) {
    const int n = a.n;
    if (!await(sm.qfull + 0, a.rows_n++, 26)) return false;
    if (a.done > 0 && !await(sm.ofree + 0, a.done - 1, 23)) return false;
#pragma unroll 1
    for (int j = 0; j <= n; ++j) {
      if (j > 0) {
        if (!await(sm.full + at.slot, at.turn, 21) || !await(sm.pfull + 0, a.tiles++, 22)) return false;
        tc_fence_after();
        pv<0>(at.slot, j == 1);
        mma_commit(sm.empty + at.slot);
        at.next();
      }
      if (j < n) {
        if (!await(sm.full + at.slot, at.turn, 25)) return false;
        tc_fence_after();
        qk<0>(at.slot);
        mma_commit(sm.empty + at.slot);
        at.next();
      }
    }
    mma_commit(sm.qfree + 0);
    mma_commit(sm.odone + 0);
    ++a.done;
    return true;
  }

  template <int S>
  __device__ __forceinline__ void lane_step(MmaSlot& s) {
    if (s.pend) {
      const uint32_t vs = at.slot;
      wait(sm.full + vs, at.turn, 21);
      at.next();
      wait(sm.pfull + S, s.tiles++, 22);
      const bool first = s.j == 1;
      if (first && s.done > 0) wait(sm.ofree + S, s.done - 1, 23);
      if (!ok) return;
      tc_fence_after();
      pv<S>(vs, first);
      mma_commit(sm.empty + vs);
      if (s.j == s.n) {
        mma_commit(sm.odone + S);
        ++s.done;
      }
      s.pend = false;
    }
    int share;
    while (ok && !s.fin && s.j == s.n) take<S>(s, &share);
    if (!ok || s.fin) return;
    const uint32_t ks = at.slot;
    wait(sm.full + ks, at.turn, 25);
    at.next();
    if (s.j == 0) wait(sm.qfull + S, s.rows_n++, 26);
    if (!ok) return;
    tc_fence_after();
    qk<S>(ks);
    ++s.j;
    if (s.j == s.n) mma_commit(sm.qfree + S);
    mma_commit(sm.empty + ks);
    s.pend = true;
  }

  __device__ __forceinline__ void run() {
    MmaSlot a, b;
    a.n = a.j = b.n = b.j = 0;
    a.seen = a.done = a.tiles = a.rows_n = 0;
    b.seen = b.done = b.tiles = b.rows_n = 0;
    a.fin = b.fin = a.pend = b.pend = false;
    // pair pieces come first, both slots told of each
    int share = 0;
    for (;;) {
      while (ok && !a.fin && a.n == 0) take<0>(a, &share);
      if (!ok || a.fin || share == 0) break;
      int other;
      take<1>(b, &other);
      if (ok) ok = share == 1 ? pair_piece(a, b) : single_piece(a);
      a.n = b.n = a.j = b.j = 0;
    }
#pragma unroll 1
    while (ok && !(a.fin && b.fin && !a.pend && !b.pend)) {
      lane_step<0>(a);
      lane_step<1>(b);
    }
    if (!ok) {
      // the MMAs issued so far complete before TMEM is freed
      volatile int no_abort = 0;
      mma_commit(sm.drain);
      mbar_wait(sm.drain, 0, &no_abort, kWaitLimitNs);
    }
  }
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
  const Smem<D> sm(smem);
  volatile int* abort_flag = sm.abort_flag;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = p.Hq / p.Hkv;

  if (threadIdx.x == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(sm.full + i, 1);
      mbar_init(sm.empty + i, 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(sm.sfull + s, 1);
      mbar_init(sm.pfull + s, 4);
      mbar_init(sm.odone + s, 1);
      mbar_init(sm.ofree + s, 4);
      mbar_init(sm.qfull + s, 1);
      mbar_init(sm.qfree + s, 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(sm.pieced + i, 1);
      mbar_init(sm.unpieced + i, 5);
      mbar_init(sm.fixset + i, 1);
      mbar_init(sm.fixdone + i, 1);
      mbar_init(sm.raw + i, 1);
    }
    mbar_init(sm.drain, 1);
    *abort_flag = 0;
    mbar_fence_init();
  }
  // a kernel that starts behind this one may then count on what this one waited for
  grid_wait();
  grid_release();
  if (warp == 1) {
    tmem_alloc(sm.tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  if (!kList)
    make_plan<kThreads / 32, 2>(p, sm.plan, reinterpret_cast<long long*>(smem + L::kOffScan),
              reinterpret_cast<int*>(smem + L::kOffScan + 12 * 8));
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *sm.tmem_slot;

  if (warp == 0) {
    if (lane == 0) {
      tma_prefetch_desc(&tm_q);
      tma_prefetch_desc(&tm_qs);
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
    }
    Producer<D, kList> producer(p, &tm_q, &tm_qs, &tm_k, &tm_v, sm, lane);
    producer.run();
  } else if (warp == 1) {
    if (lane == 0) {
      Issuer<D> issuer(sm, tmem);
      issuer.run();
    }
  } else if (warp == 2) {
    // ---------------------------------------------------------------- clearing
    // Value rows behind the keys that count hold anything, NaN included, and
    // P = 0 times NaN is not 0; halves that were not loaded hold older tiles.
    for (uint32_t i = 0;; ++i) {
      const uint32_t fi = i & 3;
      if (!wait_all(sm.fixset + fi, (i / 4) & 1, abort_flag, 31)) break;
      const int slot = sm.fixes[fi].slot, v0 = sm.fixes[fi].v0, v1 = sm.fixes[fi].v1;
      if (slot < 0) break;
      if (!wait_all(sm.raw + fi, (i / 4) & 1, abort_flag, 32)) break;
      uint8_t* base = sm.ring + slot * L::kTile;
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {
        const int v = half ? v1 : v0;
#pragma unroll 1
        for (int i = lane; i < (64 - v) * (D / 8); i += 32) {
          const int r = v + i / (D / 8), ch = i % (D / 8);
          *reinterpret_cast<uint4*>(base + half * (L::kTile / 2) + (r >> 3) * L::kGroup + (ch >> 3) * 1024 + (r & 7) * 128 +
                                    (ch & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
        }
      }
      fence_proxy_async_smem();  // these stores before the tensor core's reads
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(sm.full + slot);
        mbar_arrive(sm.fixdone + fi);
      }
    }
  } else if (warp >= 4) {
    // ---------------------------------------------------------------- softmax and results
    const int s = (warp - 4) >> 2, quarter = warp & 3;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t tS = tmem + s * 128 + lane_off, tO = tmem + 256 + s * 128 + lane_off;
    const int r = quarter * 32 + lane, rtok = r / G, rg = r - rtok * G;
    uint32_t tiles = 0, done = 0;
    bool ok = true;
    for (uint32_t i = 0; ok; ++i) {
      const Piece& d = sm.pieces[s * 2 + (i & 1)];
      if (!wait_all(sm.pieced + s * 2 + (i & 1), (i / 2) & 1, abort_flag, 41)) break;
      const int n = d.n, share = d.share, ntok = d.ntok, h = d.h, dst = d.dst;
      const int rows = share == 2 && s == 1 ? 0 : ntok * G;
      const bool live = r < rows, on = quarter * 32 < rows;  // this row, some row of the warp
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
            if (!wait_all(sm.sfull + s, tiles & 1, abort_flag, 42)) {
              ok = false;
              break;
            }
            ++tiles;
            tc_fence_after();
            if (on) {
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
              const RowTile t = !whole || __any_sync(0xffffffffu, M == -INFINITY) ? rows_first(tS, vis, c, M)
                                                                                  : rows_tile(tS, c, M, live);
              const bool moved = live && t.M != M;
              const float a = !moved ? 1.f : (M == -INFINITY ? 0.f : ex2_approx(M - t.M));
              l = l * a + t.sum;
              if (j > 0 && __any_sync(0xffffffffu, moved && M != -INFINITY)) {
                // O holds the sum through the tile before: its P V completed before these scores were formed
                const float f = moved && M != -INFINITY ? a : 1.f;
                const float2 a2 = make_float2(f, f);
#pragma unroll 1
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
            if (lane == 0) mbar_arrive(sm.pfull + s);
          }
          if (!ok) break;
          if (!wait_all(sm.odone + s, done & 1, abort_flag, 43)) break;
          ++done;
          tc_fence_after();
        }
        // l is 0 where nothing was seen; NaN stays NaN
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const float lse2 = l == 0.f ? -INFINITY : M + __log2f(l);
        if (on) {
#pragma unroll 1
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
#pragma unroll
                for (int x = 0; x < 4; ++x) st_global_v8(part + cc * 32 + 8 * x, w + 8 * x);  // whole sectors
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
          if (lane == 0) mbar_arrive(sm.ofree + s);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(sm.unpieced + s * 2 + (i & 1));
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
template <int D>
__global__ void __launch_bounds__(32 * kJoinWarps) join_ranges_kernel(const __grid_constant__ RowsParams p, int grid, int lanes) {
  grid_release();
  const int row = blockIdx.x * kJoinWarps + (threadIdx.x >> 5);
  const int G = p.Hq / p.Hkv;
  const int tok = row / p.Hq, hq = row - tok * p.Hq, h = hq / G, g = hq - h * G;
  const int b = tok / p.Nq, i = tok - b * p.Nq;
  grid_wait();
  if (row >= p.B * p.Nq * p.Hq) return;
  const long long total = p.sums[p.B], pair_total = p.sums[p.B + 1];
  const int nt = tiles_of(static_cast<int>(p.sums[p.B + 2]));
  Join s = {-INFINITY, 0.f};
  float acc[D / 32];
#pragma unroll
  for (int x = 0; x < D / 32; ++x) acc[x] = 0.f;
  // pieces of the prefix, then of the sequence's own keys: place = base + (number) * rows
  long long base0 = 0, base1 = 0;
  int n0 = 0, n1 = 0, rows0 = 256;
  if (nt > 0) {
    const int rt = tok / p.tile_tokens;
    const int unit = p.pairs ? h * p.pairs + (rt >> 1) : h;
    const long long a = static_cast<long long>(unit) * nt, all = p.pairs ? pair_total : total;
    const int runs = p.pairs ? grid : lanes, first = run_of(all, runs, a);
    n0 = run_of(all, runs, a + nt - 1) - first + 1;
    if (!p.pairs) rows0 = p.unit_rows;
    base0 = p.pairs ? (static_cast<long long>(first) + unit) * 256 + (rt & 1) * 128 + (tok - rt * p.tile_tokens) * G + g
                    : p.pair_rows + (static_cast<long long>(first) + unit) * p.unit_rows + tok * G + g;
  }
  const int own = own_tiles(p, b);
  if (own > 0) {
    const int rt = i / p.own_tokens, u = h * p.own_rt + rt;
    const long long a = p.sums[b] + static_cast<long long>(u) * own;
    const int first = run_of(total, lanes, a);
    n1 = run_of(total, lanes, a + own - 1) - first + 1;
    const long long unit = static_cast<long long>(b) * p.Hkv * p.own_rt + u + (p.pairs ? 0 : p.Hkv);
    base1 = p.pair_rows + (first + unit) * p.unit_rows + (i - rt * p.own_tokens) * G + g;
  }
  join<D>(p, n0 + n1,
          [&](int x) {
            return x < n0 ? base0 + static_cast<long long>(x) * rows0 : base1 + static_cast<long long>(x - n0) * p.unit_rows;
          },
          s, acc);
  write_row<D>(p, tok, hq, s, acc);
}

// Units of listed blocks that more than one lane computed.
template <int D>
__global__ void __launch_bounds__(32 * kJoinWarps) join_lists_kernel(const __grid_constant__ RowsParams p, int lanes) {
  grid_depends();
  const int G = p.Hq / p.Hkv;
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
  // place 2 lane, or 2 lane + 1 where the lane started in the unit before
  const int second = run_start(total, lanes, first) < a ? 1 : 0;
  join<D>(p, last - first + 1,
          [&](int x) { return static_cast<long long>(2 * (first + x) + (x == 0 ? second : 0)) * p.unit_rows + g; }, s, acc);
  const int per = p.Hkv * p.Nq, u = whole + cu;
  const int b = u / per, x = u - b * per, h = x / p.Nq;
  write_row<D>(p, b * p.Nq + x - h * p.Nq, h * G + g, s, acc);
}

template <int D, bool kList>
cudaError_t launch_wide(const RowsParams& p, const CUtensorMap& tm_q, const CUtensorMap& tm_qs, const CUtensorMap& tm_k,
                        const CUtensorMap& tm_v, int grid, cudaStream_t stream) {
  using L = Layout<D>;
  auto kern = rows_kernel<D, kList>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kAlloc);
  if (e != cudaSuccess) return e;
  return launch_dependent(kern, dim3(grid), kThreads, L::kAlloc, stream, tm_q, tm_qs, tm_k, tm_v, p);
}

// Lane work goes to few_rows_sm103.cu where its units have few rows.
template <int D>
cudaError_t launch_d(RowsParams p, const CUtensorMap& tm_q, const CUtensorMap& tm_qs, const CUtensorMap& tm_k,
                     const CUtensorMap& tm_v, cudaStream_t stream) {
  int dev = 0, n_sm = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  int grid = n_sm < kRowsCtas ? n_sm : kRowsCtas;
  const int G = p.Hq / p.Hkv;
  const bool few = p.unit_rows <= kFewRows;
  if (p.blocks) {
    const long long tiles = static_cast<long long>(p.B) * p.Nq * p.Hkv * ((p.n_sel + 1) / 2);
    if (tiles < grid) grid = static_cast<int>(tiles);
    e = few ? launch_few_rows(p, tm_qs, tm_k, tm_v, grid, false, stream)
            : launch_wide<D, true>(p, tm_q, tm_qs, tm_k, tm_v, grid, stream);
    if (e != cudaSuccess) return e;
    const int lanes = few ? grid : 2 * grid;
    const int units = p.B * p.Nq * p.Hkv, cut = units - units / lanes * lanes;
    if (cut == 0) return e;
    return launch_dependent(join_lists_kernel<D>, dim3((cut * G + kJoinWarps - 1) / kJoinWarps), 32 * kJoinWarps, 0,
                            stream, p, lanes);
  }
  p.only_pairs = few ? 1 : 0;
  if (p.pairs || !few) e = launch_wide<D, false>(p, tm_q, tm_qs, tm_k, tm_v, grid, stream);
  if (e == cudaSuccess && few) e = launch_few_rows(p, tm_qs, tm_k, tm_v, grid, p.pairs > 0, stream);
  if (e != cudaSuccess) return e;
  const long long rows = static_cast<long long>(p.B) * p.Nq * p.Hq;
  return launch_dependent(join_ranges_kernel<D>, dim3(static_cast<unsigned>((rows + kJoinWarps - 1) / kJoinWarps)),
                          32 * kJoinWarps, 0, stream, p, grid, few ? grid : 2 * grid);
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

cudaError_t status_word_wide_rows(uint32_t** at) { return cudaGetSymbolAddress(reinterpret_cast<void**>(at), g_rows_status); }

}  // namespace attn

// Attention of up to 32 query rows that read the same keys, over a paged bf16
// cache, for sm_103a: the new tokens of one sequence with a group's heads, those
// of a small batch on its shared prefix, or one token's heads on listed blocks.
//
// With few rows the keys take the MMA's M and the rows its N:
//     S^T [128 keys x N]  = K Q^T            (A: the K tile, B: Q, K-major)
//     O^T [d x N]        += V^T P^T          (A: the V tile, M-major, B: P^T)
// Both products of a tile take as long as the tensor core needs to read the
// tile from shared memory, whatever the rows: 1024 cycles for 128 keys of d = 128,
// 1100 with all that is around it, while the tile's 64 KB take 1.4 us to arrive from
// memory.  Bound by memory: 16 tokens of 32 heads on 64 listed blocks, 8 KV heads of
// d = 128, read 269 MB in 50.4 us, 5.3 TB/s.  With the rows in M (rows_sm103.cu) that
// takes 60.4 us.
//
// R, the rows that the softmax handles: 4, 8, 16 or 32.  The case above, us by R
// (by the rows in M):
//      4 rows   50.4 (4)   51.4 (8)   54.4 (16)   54.8 (32)   60.4
//      8 rows              52.1       55.1        55.4        60.9
//     16 rows                         55.8        56.1        61.4
//     32 rows                                     58.8        63.6
//
// The softmax has a thread for each key: its N scores from Tensor Memory, p to
// shared memory as the next product's operand, a part of each row's sum of p in
// its registers until the piece ends.  A row's exponent reference M is the
// largest score of its first tile; it moves (and O^T is rescaled in Tensor Memory)
// only where x - M passes 8, on which the four warps vote once a tile, so that
// p = 2^(x - M) stays below 2^8 and sums of p v have nearly all of fp32's range (with
// p up to 2^96 values from 2^32 on passed it).
//
// The work is that of the lanes of rows_sm103.cu: an equal run of (unit, key
// tile) for each CTA, pieces joined by the joining kernels there.  Scores, P,
// rows and O^T are held twice, so that neither a tile nor a piece waits for the
// one before to end.
//
// Warps: 0 loader of K, 1 and 3 issuers of the two products, 2 clears value rows,
// 4-7 (and 8-11 with more than 16 rows) softmax and results, then the loader of V
// and the planner (pieces and their pages).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "launch.h"
#include "ptx.cuh"
#include "rows_plan.cuh"

namespace attn {
namespace {

constexpr int kPieces = 4;  // pieces told ahead

struct Piece {
  int n;           // key tiles; -1: no more work
  int h;           // KV head
  int tok0, ntok;  // first token, tokens
  int key0, keys;  // ranges: position of the first key, keys from there on
  int all;         // ranges: every row sees all of them
  int dst;         // piece number, -1: the result itself
  int row;         // table row of the keys
  const int* list;  // lists: the entries, `count` of them; the token sees `seen` keys
  int count, seen;
  int part;        // keys seen of the blocks marked in some[]
  uint32_t full[kMaskWords], some[kMaskWords];  // lists: blocks seen whole, seen in part
  int group[32];   // the first 32 blocks, as groups of 8 keys of the pool
};

// R rows: 4, 8, 16 or 32.
template <int D, int R>
struct Layout {
  static constexpr int kN = R < 16 ? 16 : R;  // 16: the least that M = 128 takes
  // Softmax groups of four warps, each with kRows of the rows: the code is that of
  // 16 rows at most (one group with 32 rows a thread took 9000 cycles a tile: its
  // code no longer stayed in the instruction cache).
  static constexpr int kRows = R < 16 ? R : 16, kGroups = R / kRows;
  static constexpr int kValueWarp = 4 + 4 * kGroups, kPlanWarp = kValueWarp + 1, kWarps = kPlanWarp + 1;
  static constexpr int kTile = 128 * D * 2;
  // tiles: groups of 8 keys, each with its D / 64 blocks of 8 rows of 128 B
  static constexpr int kGroup = D / 64 * 1024;
  static constexpr int kKs = 3 * (128 / D), kVs = R == 32 && D == 128 ? 2 : kKs;  // K and V tiles held
  static constexpr int kQ = kN * D * 2;  // [D / 64][N][128 B]
  static constexpr int kP = kN * 256;    // [2][N][128 B]
  static constexpr int kOffV = kKs * kTile;
  static constexpr int kOffQ = kOffV + kVs * kTile;  // behind V: with d = 64 the product's M reads on 1 KB past a tile
  static constexpr int kOffP = kOffQ + 2 * kQ;
  static constexpr int kOffPiece = kOffP + 2 * kP;
  static constexpr int kOffBar = kOffPiece + kPieces * static_cast<int>(sizeof(Piece));
  static constexpr int kNumBars = 2 * kKs + 2 * kVs + 7 * 2 + 2 * kPieces + 3 * 4 + 2;
  static constexpr int kOffFix = kOffBar + 8 * kNumBars;
  static constexpr int kOffPlan = (kOffFix + 4 * static_cast<int>(sizeof(Fix)) + 15) & ~15;
  static constexpr int kOffScan = kOffPlan + static_cast<int>(sizeof(Plan));
  static constexpr int kOffRed = kOffScan + kWarps * 8 + 2 * kWarps * 4;  // [4][R] floats
  static constexpr int kOffRow = kOffRed + 4 * R * 4;                   // [3][R] floats
  static constexpr int kOffLim = kOffRow + 3 * R * 4;                   // [R] ints
  static constexpr int kOffMisc = kOffLim + R * 4;
  static constexpr int kBytes = kOffMisc + 32;
  static constexpr int kAlloc = kBytes + 1024;  // slack to align the base to 1024 B
  static constexpr uint32_t kTmem = 4 * kN;     // S^T twice, O^T twice
};
static_assert(Layout<128, 16>::kAlloc <= 232448 && Layout<64, 16>::kAlloc <= 232448 && Layout<128, 32>::kAlloc <= 232448 &&
                  Layout<64, 32>::kAlloc <= 232448, "shared memory of a CTA");

template <int D, int R>
struct Smem {
  uint8_t *k, *v, *q, *ps;
  Piece* pieces;
  uint64_t* kfull;     // [kKs] K slot holds its tile
  uint64_t* kempty;    // [kKs] K slot read
  uint64_t* vfull;     // [kVs] V slot holds its tile
  uint64_t* vempty;    // [kVs] V slot read
  uint64_t* sfull;     // [2] scores complete
  uint64_t* pfull;     // [2] P written (4 warps)
  uint64_t* pvdone;    // [2] a tile's P V complete
  uint64_t* odone;     // [2] a piece's last P V complete
  uint64_t* ofree;     // [2] a piece's O read (4 warps)
  uint64_t* qfull;     // [2] rows loaded
  uint64_t* qfree;     // [2] a piece's last Q K^T complete
  uint64_t* pieced;    // [kPieces] piece told
  uint64_t* unpieced;  // [kPieces] piece done with (loaders, issuers, 4 softmax warps)
  uint64_t* fixset;    // [4] clearing asked for
  uint64_t* fixdone;   // [4] done
  uint64_t* raw;       // [4] value tile to be cleared landed
  uint64_t* drain;     // [2] after an abort: the MMAs that an issuer issued so far completed
  Fix* fixes;
  Plan* plan;
  // of each softmax group, one after the other:
  float* red;  // [4][kRows] of its warps
  float* row;  // [kRows] references, [2][kRows] factors of its rows
  int* lim;    // [kRows] keys of the piece that a row sees
  uint32_t* tmem_slot;
  volatile int* abort_flag;
  volatile int* gone;  // [2][2] a warp of the softmax group gave up (by the tile's parity)
  __device__ __forceinline__ explicit Smem(uint8_t* base) {
    using L = Layout<D, R>;
    k = base;
    v = base + L::kOffV;
    q = base + L::kOffQ;
    ps = base + L::kOffP;
    pieces = reinterpret_cast<Piece*>(base + L::kOffPiece);
    kfull = reinterpret_cast<uint64_t*>(base + L::kOffBar);
    kempty = kfull + L::kKs;
    vfull = kempty + L::kKs;
    vempty = vfull + L::kVs;
    sfull = vempty + L::kVs;
    pfull = sfull + 2;
    pvdone = pfull + 2;
    odone = pvdone + 2;
    ofree = odone + 2;
    qfull = ofree + 2;
    qfree = qfull + 2;
    pieced = qfree + 2;
    unpieced = pieced + kPieces;
    fixset = unpieced + kPieces;
    fixdone = fixset + 4;
    raw = fixdone + 4;
    drain = raw + 4;
    fixes = reinterpret_cast<Fix*>(base + L::kOffFix);
    plan = reinterpret_cast<Plan*>(base + L::kOffPlan);
    red = reinterpret_cast<float*>(base + L::kOffRed);
    row = reinterpret_cast<float*>(base + L::kOffRow);
    lim = reinterpret_cast<int*>(base + L::kOffLim);
    tmem_slot = reinterpret_cast<uint32_t*>(base + L::kOffMisc);
    abort_flag = reinterpret_cast<volatile int*>(base + L::kOffMisc + 4);
    gone = reinterpret_cast<volatile int*>(base + L::kOffMisc + 8);
  }
};

// ---------------------------------------------------------------------------
// Planner: a warp that works out the pieces, up to kPieces ahead, with their first
// 32 blocks looked up in the table (a lane each), so that the loaders have no
// chain of loads of their own between two pieces.
template <int D, int R, bool kList>
struct Planner {
  const RowsParams& p;
  const Smem<D, R>& sm;
  const int lane;
  uint32_t told = 0;
  bool ok = true;
  // the CTA's run
  long long left, unit;  // tiles left (lists: of the cut units); lists: next whole unit
  int b, hh, rt, t;      // ranges: where it stands

  __device__ __forceinline__ Planner(const RowsParams& p_, const Smem<D, R>& sm_) : p(p_), sm(sm_), lane(threadIdx.x & 31) {}

  // Next piece; false: no more, or given up.
  __device__ __forceinline__ bool next_piece() {
    const int lanes = gridDim.x, l = blockIdx.x;
    if (told >= kPieces) ok = wait_all(sm.unpieced + told % kPieces, (told / kPieces - 1) & 1, sm.abort_flag, 13);
    if (!ok) return false;
    Piece& d = sm.pieces[told % kPieces];
    uint64_t* bar = sm.pieced + told % kPieces;
    ++told;
    int n = -1, h = 0, tok0 = 0, ntok = 0, key0 = 0, end = 0, all = 0, dst = -1, row = 0, count = 0, seen = 0;
    const int* list = nullptr;
    if (kList) {
      const int units = p.B * p.Nq * p.Hkv, unit_tiles = (p.n_sel + 1) >> 1;
      const int whole = units / lanes * lanes;
      long long u = -1;
      int t0 = 0, nt = unit_tiles;
      if (unit < whole) {
        u = unit;
        unit += lanes;
      } else if (left > 0) {
        const long long cut = static_cast<long long>(units - whole) * unit_tiles;
        const long long first = run_start(cut, lanes, l), x = run_start(cut, lanes, l + 1) - left;
        const int cu = static_cast<int>(quotient(x, unit_tiles));
        u = whole + cu;
        t0 = static_cast<int>(x - static_cast<long long>(cu) * unit_tiles);
        nt = static_cast<int>(min(static_cast<long long>(unit_tiles - t0), left));
        if (nt < unit_tiles) dst = 2 * l + (x > first ? 1 : 0);
        left -= nt;
      }
      if (u >= 0) {
        // units by sequence, head, token: neighbours read the same head's keys
        const int per = p.Hkv * p.Nq, ui = static_cast<int>(u);
        row = ui / per;
        const int r = ui - row * per;
        h = r / p.Nq;
        const int i = r - h * p.Nq;
        tok0 = row * p.Nq + i;
        ntok = 1;
        list = p.blocks + (static_cast<long long>(tok0) * p.Hkv + h) * p.n_sel + 2 * t0;
        count = min(p.n_sel - 2 * t0, 2 * nt);
        const int len = clamped_len(p, row);
        if (lane == 0 && h == 0 && i == 0 && t0 == 0 && len != p.seqlens[row]) record(1, kDevBadSeqlen);
        seen = max(0, len - p.Nq + i + 1);
        // which of them are seen; the last one that is ends the piece
        int last = -1;
        for (int w = 0; w < (count + 31) >> 5; ++w) {
          const int e = 32 * w + lane;
          const int blk = e < count ? list[e] : -1;
          int v = 0;
          if (blk >= 0) {
            if (blk >= p.max_blocks * (p.page_size / 64))
              record(3, kDevBadPage);
            else
              v = min(64, seen - blk * 64);
          }
          if (w == 0) d.group[lane] = v > 0 ? pool_group(p, row, blk) : 0;
          const uint32_t any = __ballot_sync(0xffffffffu, v > 0), full = __ballot_sync(0xffffffffu, v == 64);
          const uint32_t some = any & ~full;
          if (lane == 0) {
            d.full[w] = full;
            d.some[w] = some;
          }
          if (some) {
            const int part = __shfl_sync(0xffffffffu, v, __ffs(some) - 1);  // the same for all of them
            if (lane == 0) d.part = part;
          }
          if (any) last = 32 * w + 31 - __clz(any);
        }
        n = (last + 2) >> 1;
      }
    } else if (left > 0) {
      int len = b < 0 ? 0 : clamped_len(p, b);
      while (b >= 0 && len <= p.shared_len) len = clamped_len(p, ++b);  // a sequence with keys of its own is ahead
      int nt, rts, u;
      h = hh;
      if (b < 0) {
        end = sm.plan->prefix_end;
        key0 = 128 * t;
        nt = tiles_of(end);
        all = sm.plan->all_see >= end;
        rts = 1;
        u = hh;
        ntok = p.B * p.Nq;
      } else {
        end = len;
        key0 = p.shared_len + 128 * t;
        row = b;
        nt = tiles_of(len - p.shared_len);
        all = p.Nq == 1;
        rts = p.own_rt;
        u = (b * p.Hkv + hh) * rts + rt + (p.pairs ? 0 : p.Hkv);
        tok0 = b * p.Nq + rt * p.own_tokens;
        ntok = min(p.own_tokens, p.Nq - rt * p.own_tokens);
      }
      dst = l + u;
      n = static_cast<int>(min(static_cast<long long>(nt - t), left));
      left -= n;
      const int key = key0 + 64 * lane;
      d.group[lane] = key < end && lane < 2 * n ? pool_group(p, row, key >> 6) : 0;
      t += n;
      if (t == nt) {
        t = 0;
        if (++rt == rts) {
          rt = 0;
          if (++hh == p.Hkv) {
            hh = 0;
            ++b;
          }
        }
      }
    }
    if (lane == 0) {
      d.n = n;
      d.h = h;
      d.tok0 = tok0;
      d.ntok = ntok;
      d.key0 = key0;
      d.keys = end - key0;
      d.all = all;
      d.dst = dst;
      d.row = row;
      d.list = list;
      d.count = count;
      d.seen = seen;
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
    return n >= 0;
  }

  __device__ __forceinline__ void run() {
    const int lanes = gridDim.x, l = blockIdx.x;
    if (kList) {
      const int units = p.B * p.Nq * p.Hkv;
      const long long cut = static_cast<long long>(units - units / lanes * lanes) * ((p.n_sel + 1) >> 1);
      unit = l;
      left = run_start(cut, lanes, l + 1) - run_start(cut, lanes, l);
    } else {
      const long long total = sm.plan->total;
      left = run_start(total, lanes, l + 1) - run_start(total, lanes, l);
      if (left > 0) {
        b = sm.plan->lane_b[0];
        const int nt = b < 0 ? tiles_of(sm.plan->prefix_end) : own_tiles(p, b), rts = b < 0 ? 1 : p.own_rt;
        const long long x = sm.plan->lane_at[0];
        const int u = static_cast<int>(quotient(x, nt));
        hh = u / rts;
        rt = u - hh * rts;
        t = static_cast<int>(x - static_cast<long long>(u) * nt);
      }
    }
#pragma unroll 1
    while (next_piece()) {
    }
  }
};

// Loaders: a warp for K tiles (and a piece's rows) and one for V tiles; lane 0
// waits and issues.  (One warp for both took 770 cycles a tile and operand.)
template <int D, int R, bool kList, bool kV>
struct Loader {
  using L = Layout<D, R>;
  const RowsParams& p;
  const CUtensorMap *tm, *tm_q;
  const Smem<D, R>& sm;
  const int lane;
  RingAt<kV ? L::kVs : L::kKs> at;
  uint32_t fix_n = 0, rows_n = 0;
  bool ok = true;  // lane 0's view until `agree`

  __device__ __forceinline__ Loader(const RowsParams& p_, const CUtensorMap* tm_, const CUtensorMap* q, const Smem<D, R>& sm_)
      : p(p_), tm(tm_), tm_q(q), sm(sm_), lane(threadIdx.x & 31) {}

  __device__ __forceinline__ void wait(uint64_t* bar, uint32_t parity, uint32_t site) {
    if (ok) ok = wait_one(bar, parity & 1, sm.abort_flag, site);
  }
  __device__ __forceinline__ bool agree() {
    ok = __shfl_sync(0xffffffffu, static_cast<int>(ok), 0) != 0;
    return ok;
  }
  // this lane's block of blocks 32 i .. 32 i + 31 of a piece
  __device__ __forceinline__ int look_up(const Piece& d, int i) {
    if (kList) {
      const uint32_t seen = d.full[i] | d.some[i];
      return seen >> lane & 1u ? pool_group(p, d.row, d.list[32 * i + lane]) : 0;
    }
    const int key = d.key0 + 64 * (32 * i + lane);
    return key < d.key0 + d.keys && 32 * i + lane < 2 * d.n ? pool_group(p, d.row, key >> 6) : 0;
  }
  // a tile into the next slot: its blocks g0, g1, of which v0 and v1 keys count
  __device__ __forceinline__ void load(int g0, int g1, int v0, int v1, int head) {
    uint64_t* full = (kV ? sm.vfull : sm.kfull) + at.slot;
    if (at.turn > 0) wait((kV ? sm.vempty : sm.kempty) + at.slot, at.turn - 1, 11);
    if (!ok) return;
    uint8_t* dst = (kV ? sm.v : sm.k) + at.slot * L::kTile;
    if (v0 == 64 && v1 == 64) {
      mbar_arrive_expect_tx(full, L::kTile);
      tma_load_5d(dst, tm, full, 0, 0, 0, g0, head);
      tma_load_5d(dst + L::kTile / 2, tm, full, 0, 0, 0, g1, head);
    } else {
      const uint32_t fi = fix_n & 3;
      uint64_t* done = kV ? sm.raw + fi : full;
      if (kV) {
        if (fix_n >= 4) wait(sm.fixdone + fi, fix_n / 4 - 1, 12);
        if (!ok) return;
        sm.fixes[fi].slot = static_cast<int>(at.slot);
        sm.fixes[fi].v0 = v0;
        sm.fixes[fi].v1 = v1;
      }
      if (v0 || v1)
        mbar_arrive_expect_tx(done, v0 && v1 ? L::kTile : L::kTile / 2);
      else
        mbar_arrive(done);
      if (v0) tma_load_5d(dst, tm, done, 0, 0, 0, g0, head);
      if (v1) tma_load_5d(dst + L::kTile / 2, tm, done, 0, 0, 0, g1, head);
      if (kV) {
        mbar_arrive(sm.fixset + fi);
        ++fix_n;
      }
    }
    at.next();
  }
  __device__ __forceinline__ void run() {
    for (uint32_t i = 0;; ++i) {
      const Piece& d = sm.pieces[i % kPieces];
      if (lane == 0) wait(sm.pieced + i % kPieces, i / kPieces, 15);
      if (!agree()) break;
      const int n = d.n, h = d.h;
      if (n < 0) break;
      if (!kV && n > 0 && lane == 0) {
        const uint32_t buf = rows_n & 1;
        if (rows_n >= 2) wait(sm.qfree + buf, rows_n / 2 - 1, 14);
        if (ok) {
          mbar_arrive_expect_tx(sm.qfull + buf, static_cast<uint32_t>(p.unit_tokens * (p.Hq / p.Hkv) * D * 2));
#pragma unroll
          for (int c = 0; c < D / 64; ++c)
            tma_load_4d(sm.q + buf * L::kQ + c * (L::kN * 128), tm_q, sm.qfull + buf, c * 64, 0, h, d.tok0);
          ++rows_n;
        }
      }
      int blk = d.group[lane], next = 0;
      const int keys = d.keys, part = d.part;
#pragma unroll 1
      for (int j = 0; j < n; ++j) {
        if ((j & 15) == 0 && j > 0) blk = next;
        const int e = 2 * (j & 15);
        const int g0 = __shfl_sync(0xffffffffu, blk, e), g1 = __shfl_sync(0xffffffffu, blk, e + 1);
        if (lane == 0) {
          int v0, v1;
          if (kList) {
            const uint32_t f = d.full[j >> 4] >> e, m = d.some[j >> 4] >> e;
            v0 = f & 1u ? 64 : (m & 1u ? part : 0);
            v1 = f & 2u ? 64 : (m & 2u ? part : 0);
          } else {
            v0 = min(64, keys - 128 * j);
            v1 = max(0, min(64, keys - 128 * j - 64));
          }
          load(g0, g1, v0, v1, h);
        }
        if ((j & 15) == 4 && (j | 15) + 1 < n) next = look_up(d, (j >> 4) + 1);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(sm.unpieced + i % kPieces);
    }
    if (lane != 0) return;
    if (kV && ok) {
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
#pragma unroll 1
    for (uint32_t i = 0; i < 2 && i < rows_n; ++i) mbar_wait(sm.qfull + i, (rows_n - 1 - i) / 2 & 1, &no_abort, kWaitLimitNs);
#pragma unroll 1
    for (uint32_t i = 0; i < 4 && i < fix_n; ++i) mbar_wait(sm.raw + i, (fix_n - 1 - i) / 4 & 1, &no_abort, kWaitLimitNs);
#pragma unroll 1
    for (uint32_t i = 0; i < (kV ? L::kVs : L::kKs); ++i) {
      const uint32_t turns = at.turn + (i < at.slot ? 1 : 0);
      if (turns > 0) mbar_wait((kV ? sm.vfull : sm.kfull) + i, (turns - 1) & 1, &no_abort, kWaitLimitNs);
    }
  }
};

// ---------------------------------------------------------------------------
// Issuers of the two products, a thread each: their instructions between the
// products overlap (one thread for both took 2100 cycles a tile, of which the
// tensor core was busy half).
template <int D, int R>
struct Issuer {
  using L = Layout<D, R>;
  static constexpr uint32_t kN = L::kN;
  const Smem<D, R>& sm;
  const uint32_t tmem;
  uint32_t told = 0, piece = 0, tile = 0;  // pieces looked at, with products (before this one); tiles
  int n = 0;
  bool ok = true;

  __device__ __forceinline__ Issuer(const Smem<D, R>& sm_, uint32_t tmem_) : sm(sm_), tmem(tmem_) {}
  __device__ __forceinline__ void wait(uint64_t* bar, uint32_t parity, uint32_t site) {
    if (ok) ok = wait_one(bar, parity & 1, sm.abort_flag, site);
  }
  // tiles of the next piece, -1: no more
  __device__ __forceinline__ bool take() {
    const uint32_t at = told % kPieces;
    wait(sm.pieced + at, told / kPieces, 24);
    if (!ok) return false;
    n = *const_cast<const volatile int*>(&sm.pieces[at].n);
    mbar_arrive(sm.unpieced + at);
    ++told;
    return n >= 0;
  }
  __device__ __forceinline__ void finish(int which) {
    if (ok) return;
    // the MMAs issued so far complete before TMEM is freed
    volatile int no_abort = 0;
    mma_commit(sm.drain + which);
    mbar_wait(sm.drain + which, 0, &no_abort, kWaitLimitNs);
  }

  __device__ __forceinline__ void scores() {
    constexpr uint32_t idesc = idesc_bf16_f32(128, kN, 0);
    const uint64_t dK = sdesc_sw128(smem_u32(sm.k), 16, L::kGroup), dQ = sdesc_sw128(smem_u32(sm.q), 16, 1024);
    RingAt<L::kKs> at;
    while (take()) {
      const uint64_t q = dQ + static_cast<uint64_t>(((piece & 1) * L::kQ) >> 4);
      for (int j = 0; j < n; ++j, ++tile) {
        if (j == 0) wait(sm.qfull + (piece & 1), piece / 2, 26);
        // the tile before the last left these scores: it wrote P
        if (tile >= 2) wait(sm.pfull + (tile & 1), tile / 2 - 1, 27);
        wait(sm.kfull + at.slot, at.turn, 25);
        if (!ok) break;
        tc_fence_after();
        const uint64_t a = dK + static_cast<uint64_t>((at.slot * L::kTile) >> 4);
        const uint32_t to = tmem + (tile & 1) * kN;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_bf16_ss(to, a + (((kk >> 2) * 1024 + (kk & 3) * 32) >> 4), q + (((kk >> 2) * (kN * 128) + (kk & 3) * 32) >> 4),
                      idesc, kk > 0 ? 1u : 0u);
        mma_commit(sm.sfull + (tile & 1));
        mma_commit(sm.kempty + at.slot);
        at.next();
      }
      if (!ok) break;
      if (n > 0) mma_commit(sm.qfree + (piece++ & 1));
    }
    finish(0);
  }
  __device__ __forceinline__ void outputs() {
    // A runs along M; d = 64: M = 128 takes two 64-dim blocks, of which the second
    // (the keys behind, whatever lies there) only reaches lanes that nothing reads
    constexpr uint32_t idesc = idesc_bf16_f32(128, kN, 0) | (1u << 15);
    const uint64_t dV = sdesc_sw128(smem_u32(sm.v), 1024, L::kGroup), dP = sdesc_sw128(smem_u32(sm.ps), 16, 1024);
    RingAt<L::kVs> at;
    while (take()) {
      const uint32_t to = tmem + (2 + (piece & 1)) * kN;
      for (int j = 0; j < n; ++j, ++tile) {
        if (j == 0 && piece >= 2) wait(sm.ofree + (piece & 1), piece / 2 - 1, 23);
        wait(sm.vfull + at.slot, at.turn, 21);
        wait(sm.pfull + (tile & 1), tile / 2, 22);
        if (!ok) break;
        tc_fence_after();
        const uint64_t a = dV + static_cast<uint64_t>((at.slot * L::kTile) >> 4),
                       q = dP + static_cast<uint64_t>(((tile & 1) * L::kP) >> 4);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_bf16_ss(to, a + ((kk * 2 * L::kGroup) >> 4), q + (((kk >> 2) * (kN * 128) + (kk & 3) * 32) >> 4), idesc,
                      (j > 0 || kk > 0) ? 1u : 0u);
        mma_commit(sm.pvdone + (tile & 1));
        mma_commit(sm.vempty + at.slot);
        at.next();
      }
      if (!ok) break;
      if (n > 0) mma_commit(sm.odone + (piece++ & 1));
    }
    finish(1);
  }
};

// ---------------------------------------------------------------------------
// The first R columns of this thread's TMEM lane.
template <int R>
__device__ __forceinline__ void tmem_row(uint32_t addr, float (&x)[R]) {
  uint32_t u[R];
  if constexpr (R == 4) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3])
                 : "r"(addr));
  } else if constexpr (R == 8) {
    tmem_ld8(addr, u);
  } else {
#pragma unroll
    for (int i = 0; i < R; i += 16) tmem_ld16(addr + i, u + i);
  }
  tmem_wait_ld();
#pragma unroll
  for (int i = 0; i < R; ++i) x[i] = __uint_as_float(u[i]);
}
template <int R>
__device__ __forceinline__ void tmem_put_row(uint32_t addr, const float (&x)[R]) {
#pragma unroll
  for (int i = 0; i < R; i += 4)
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr + i), "r"(__float_as_uint(x[i])),
                 "r"(__float_as_uint(x[i + 1])), "r"(__float_as_uint(x[i + 2])), "r"(__float_as_uint(x[i + 3]))
                 : "memory");
  tmem_wait_st();
}

// Joins the warp's values of each of R rows (a power of two): by steps that halve
// the rows a lane holds, then over the lanes of a row.  Lane i returns row
// row_of(i)'s result.
template <int R, typename Op>
__device__ __forceinline__ float over_warp(const float (&x)[R], Op op) {
  const int lane = threadIdx.x & 31;
  float v[R];
#pragma unroll
  for (int r = 0; r < R; ++r) v[r] = x[r];
  int o = 16;
#pragma unroll
  for (int n = R / 2; n >= 1; n /= 2, o /= 2) {
    const bool up = lane & o;
#pragma unroll
    for (int r = 0; r < n; ++r) {
      const float give = up ? v[r] : v[r + n], keep = up ? v[r + n] : v[r];
      v[r] = op(keep, __shfl_xor_sync(0xffffffffu, give, o));
    }
  }
#pragma unroll
  for (; o > 0; o /= 2) v[0] = op(v[0], __shfl_xor_sync(0xffffffffu, v[0], o));
  return v[0];
}
// The row whose result over_warp leaves in this lane: the first step parts the
// rows by lane bit 4, the next by bit 3, and so on.
template <int R>
__device__ __forceinline__ int row_of(int lane) {
  return lane * R >> 5;
}

// The four warps of a softmax group meet; true if any thread passes true.
__device__ __forceinline__ bool group_any(int grp, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %2, 128, p;\n\tselp.b32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(x)), "r"(1 + grp)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void group_sync(int grp) { asm volatile("barrier.cta.sync %0, 128;" ::"r"(1 + grp) : "memory"); }

constexpr float kMoveLog2 = 8.f;  // a row's reference moves where a score passes it by this much

template <int D, int kR, bool kList>
struct Softmax {
  using L = Layout<D, kR>;
  static constexpr int R = L::kRows;
  const RowsParams& p;
  const Smem<D, kR>& sm;
  const uint32_t tmem;
  const int grp, lane, w4, key;  // key: of the tile (TMEM lane), and output dim
  float* const red;
  float* const row;
  int* const lim_of;
  float M[R], l[R];
  uint32_t ts = 0, piece = 0;
  bool ok = true;  // this warp's view; all leave together

  __device__ __forceinline__ Softmax(const RowsParams& p_, const Smem<D, kR>& sm_, uint32_t tmem_)
      : p(p_), sm(sm_), tmem(tmem_ + (static_cast<uint32_t>((threadIdx.x >> 5) & 3) << 21) + ((threadIdx.x >> 7) - 1) * R),
        grp((threadIdx.x >> 7) - 1), lane(threadIdx.x & 31), w4((threadIdx.x >> 5) & 3), key(threadIdx.x & 127),
        red(sm_.red + 4 * R * grp), row(sm_.row + 3 * R * grp), lim_of(sm_.lim + R * grp) {}

  __device__ __forceinline__ void wait(uint64_t* bar, uint32_t parity, uint32_t site) {
    if (ok) ok = wait_all(bar, parity & 1, sm.abort_flag, site);
  }

  // New references from this tile's largest scores; O^T and the sums so far are
  // brought to them.  s: the scores, scaled; where not `vis` they do not count.
  __device__ __forceinline__ void move(const float (&s)[R], uint32_t vis, bool first) {
    float x[R];
#pragma unroll
    for (int r = 0; r < R; ++r) x[r] = vis >> r & 1u ? s[r] : -INFINITY;
    red[w4 * R + row_of<R>(lane)] = over_warp<R>(x, [](float a, float b) { return fmaxf(a, b); });
    group_sync(grp);
    // a thread a row: its new reference and the factor of what there is (0 where nothing was seen)
    if (key < R) {
      const float mx = fmaxf(fmaxf(red[key], red[R + key]), fmaxf(red[2 * R + key], red[3 * R + key]));
      const float was = first ? -INFINITY : row[key];
      const float m = was == -INFINITY || mx - was > kMoveLog2 ? fmaxf(was, mx) : was;
      row[key] = m;
      red[key] = was == m ? 1.f : ex2_approx(was - m);  // its place was read by this thread
    }
    group_sync(grp);
#pragma unroll
    for (int r = 0; r < R; ++r) M[r] = row[r];
    if (first) return;
    wait(sm.pvdone + ((ts - 1) & 1), (ts - 1) / 2, 44);
    tc_fence_after();
    float o[R];
    const uint32_t at = tmem + (2 + (piece & 1)) * L::kN;
    tmem_row<R>(at, o);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float f = red[r];
      o[r] *= f;
      l[r] *= f;
    }
    tmem_put_row<R>(at, o);
    group_sync(grp);  // the factors are read
  }

  // Outputs of a piece, behind its last product: rows, their factors in row[R + which R ..].
  static constexpr uint32_t kNone = 0xffffffffu;
  struct Ended {
    bool on;
    int rows, tok0, h, dst;
    uint32_t which, piece;  // piece: number among those with products, kNone without
  };
  __device__ __forceinline__ void write_results(Ended& e) {
    if (!e.on) return;
    group_sync(grp);  // the factors are there
    float o[R];
    const bool any = e.piece != kNone;
    if (any) {
      wait(sm.odone + (e.piece & 1), e.piece / 2, 43);
      tc_fence_after();
      tmem_row<R>(tmem + (2 + (e.piece & 1)) * L::kN, o);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(sm.ofree + (e.piece & 1));
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float f = row[R + e.which * R + r];
      o[r] = any && f != 0.f ? o[r] * f : 0.f;
    }
    if (key < D) {
      if (e.dst >= 0) {
        float* to = p.o_part + (p.pair_rows + static_cast<long long>(e.dst) * p.unit_rows + R * grp) * D + key;
#pragma unroll
        for (int r = 0; r < R; ++r)
          if (r < e.rows) to[r * D] = o[r];
      } else {
        const int G = p.Hq / p.Hkv;
        const int skip = R * grp / G;  // tokens of the groups before
        int g = R * grp - skip * G;
        __nv_bfloat16* to =
            static_cast<__nv_bfloat16*>(p.o) + (static_cast<long long>(e.tok0 + skip) * p.Hq + e.h * G + g) * D + key;
#pragma unroll
        for (int r = 0; r < R; ++r) {
          if (r >= e.rows) break;
          *to = __float2bfloat16_rn(o[r]);
          to += D;
          if (++g == G) {  // the next token's heads of the group
            g = 0;
            to += static_cast<long long>(p.Hq - G) * D;
          }
        }
      }
    }
    e.on = false;
  }

  __device__ __forceinline__ void run() {
    const int G = p.Hq / p.Hkv;
    Ended before;
    before.on = false;
    for (uint32_t i = 0;; ++i) {
      const Piece& d = sm.pieces[i % kPieces];
      wait(sm.pieced + i % kPieces, i / kPieces, 41);
      if (group_any(grp, !ok)) return;
      const int n = d.n, h = d.h, tok0 = d.tok0, ntok = d.ntok, dst = d.dst;
      if (n < 0) break;
      const int rows = min(max(ntok * G - R * grp, 0), R);  // of this group
      int whole = 0;  // ranges: keys that all rows see
      const bool all = kList || d.all;
      if (!kList) {
        whole = d.keys;
        if (!all) {
          int lim = 0x7fffffff;
          if (key < rows) {
            const int tok = tok0 + (R * grp + key) / G, b = tok / p.Nq;
            lim = min(whole, clamped_len(p, b) - p.Nq + tok - b * p.Nq + 1 - d.key0);
            lim_of[key] = lim;
          }
          const int m = __reduce_min_sync(0xffffffffu, lim);
          if (lane == 0) red[w4] = __int_as_float(m);
          group_sync(grp);
          whole = min(min(__float_as_int(red[0]), __float_as_int(red[1])),
                      min(__float_as_int(red[2]), __float_as_int(red[3])));
          group_sync(grp);
        }
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        M[r] = -INFINITY;
        l[r] = 0.f;
      }
      for (int j = 0; j < n; ++j, ++ts) {
        wait(sm.sfull + (ts & 1), ts / 2, 42);
        tc_fence_after();
        float s[R];
        tmem_row<R>(tmem + (ts & 1) * L::kN, s);
        uint32_t vis = ~0u;  // rows that see this key
        if (kList) {
          const int e = 2 * j + (key >> 6);
          const int v = d.full[e >> 5] >> (e & 31) & 1u ? 64 : (d.some[e >> 5] >> (e & 31) & 1u ? d.part : 0);
          if ((key & 63) >= v) vis = 0;
        } else if (128 * (j + 1) > whole) {
          if (all) {
            if (128 * j + key >= whole) vis = 0;
          } else {
#pragma unroll 1
            for (int r = 0; r < rows; ++r)
              if (128 * j + key >= lim_of[r]) vis &= ~(1u << r);
          }
        }
        bool over = j == 0;
#pragma unroll
        for (int r = 0; r < R; ++r) {
          s[r] *= p.scale_log2;
          over = over || (r < rows && (vis >> r & 1u) && s[r] - M[r] > kMoveLog2);
        }
        if (!ok) sm.gone[2 * grp + (ts & 1)] = 1;
        if (group_any(grp, over || !ok)) {
          if (sm.gone[2 * grp + (ts & 1)]) return;
          move(s, vis, j == 0);
        }
        // p, to its place in the operand: rows of 128 B (64 keys), chunks of 16 B
        // exchanged by the row; the product that read this buffer is done
        if (ts >= 2) wait(sm.pvdone + (ts & 1), ts / 2 - 1, 45);
        uint8_t* to = sm.ps + (ts & 1) * L::kP + (key >> 6) * (L::kN * 128) + R * grp * 128 + (key & 7) * 2;
        const int ch = (key & 63) >> 3;
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float x = ex2_approx(s[r] - (M[r] == -INFINITY ? 0.f : M[r]));
          const float v = vis >> r & 1u ? x : 0.f;
          l[r] += v;
          *reinterpret_cast<__nv_bfloat16*>(to + r * 128 + ((ch ^ (r & 7)) << 4)) = __float2bfloat16_rn(v);
        }
        tc_fence_before();
        fence_proxy_async_smem();  // P before the tensor core's reads
        __syncwarp();
        if (lane == 0) mbar_arrive(sm.pfull + (ts & 1));
        // the piece before ended with a product that was still to come
        if (j == 0) write_results(before);
      }
      if (n == 0) write_results(before);
      // sums of the rows: over a warp's keys, then the four warps
      red[w4 * R + row_of<R>(lane)] = over_warp<R>(l, [](float a, float b) { return a + b; });
      group_sync(grp);
      // a thread a row: the factor of its outputs and its log-sum-exp; l is 0 where nothing was seen, NaN stays NaN
      if (key < rows) {
        const float sum = (red[key] + red[R + key]) + (red[2 * R + key] + red[3 * R + key]);
        const float lse2 = sum == 0.f ? -INFINITY : row[key] + __log2f(sum);
        row[R + (i & 1) * R + key] = sum == 0.f ? 0.f : 1.f / sum;
        if (dst >= 0) {
          p.lse_part[p.pair_rows + static_cast<long long>(dst) * p.unit_rows + R * grp + key] = lse2;
        } else {
          const int r = R * grp + key, tok = tok0 + r / G, b = tok / p.Nq;
          p.lse[(static_cast<long long>(b) * p.Hq + h * G + r % G) * p.Nq + tok - b * p.Nq] = lse2 * 0.6931471805599453f;
        }
      }
      before = {true, rows, tok0, h, dst, i & 1u, n > 0 ? piece : kNone};
      if (n > 0) ++piece;
      __syncwarp();
      if (lane == 0) mbar_arrive(sm.unpieced + i % kPieces);
    }
    write_results(before);
  }
};

// after_pairs: the kernel before on the stream is that of the pairs, whose CTAs
// have all passed their own wait when this one starts: nothing it reads is
// still being written, so it takes the SMs as they come free, and only ends
// after that kernel (the joining kernel waits for this one).
template <int D, int R, bool kList>
__global__ void __launch_bounds__(32 * Layout<D, R>::kWarps, 1)
    few_rows_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ RowsParams p, int after_pairs) {
  using L = Layout<D, R>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const Smem<D, R> sm(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < L::kKs; ++i) {
      mbar_init(sm.kfull + i, 1);
      mbar_init(sm.kempty + i, 1);
    }
    for (int i = 0; i < L::kVs; ++i) {
      mbar_init(sm.vfull + i, 1);
      mbar_init(sm.vempty + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(sm.sfull + i, 1);
      mbar_init(sm.pfull + i, 4 * L::kGroups);
      mbar_init(sm.pvdone + i, 1);
      mbar_init(sm.odone + i, 1);
      mbar_init(sm.ofree + i, 4 * L::kGroups);
      mbar_init(sm.qfull + i, 1);
      mbar_init(sm.qfree + i, 1);
      sm.gone[i] = sm.gone[2 + i] = 0;
    }
    for (int i = 0; i < kPieces; ++i) {
      mbar_init(sm.pieced + i, 1);
      mbar_init(sm.unpieced + i, 4 + 4 * L::kGroups);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(sm.fixset + i, 1);
      mbar_init(sm.fixdone + i, 1);
      mbar_init(sm.raw + i, 1);
    }
    mbar_init(sm.drain, 1);
    mbar_init(sm.drain + 1, 1);
    *sm.abort_flag = 0;
    mbar_fence_init();
  }
  grid_release();
  if (!after_pairs) grid_wait();
  if (warp == 1) {
    tmem_alloc(sm.tmem_slot, L::kTmem);
    tmem_relinquish();
  }
  if (!kList)
    make_plan<L::kWarps, 1>(p, sm.plan, reinterpret_cast<long long*>(smem + L::kOffScan),
                            reinterpret_cast<int*>(smem + L::kOffScan + L::kWarps * 8));
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *sm.tmem_slot;

  if (warp == 0) {
    if (lane == 0) {
      tma_prefetch_desc(&tm_q);
      tma_prefetch_desc(&tm_k);
    }
    Loader<D, R, kList, false> loader(p, &tm_k, &tm_q, sm);
    loader.run();
  } else if (warp == L::kValueWarp) {
    if (lane == 0) tma_prefetch_desc(&tm_v);
    Loader<D, R, kList, true> loader(p, &tm_v, nullptr, sm);
    loader.run();
  } else if (warp == L::kPlanWarp) {
    Planner<D, R, kList> planner(p, sm);
    planner.run();
  } else if (warp == 1) {
    if (lane == 0) {
      Issuer<D, R> issuer(sm, tmem);
      issuer.scores();
    }
  } else if (warp == 3) {
    if (lane == 0) {
      Issuer<D, R> issuer(sm, tmem);
      issuer.outputs();
    }
  } else if (warp == 2) {
    for (uint32_t i = 0;; ++i) {
      const uint32_t fi = i & 3;
      if (!wait_all(sm.fixset + fi, i / 4 & 1, sm.abort_flag, 31)) break;
      const int slot = sm.fixes[fi].slot, v0 = sm.fixes[fi].v0, v1 = sm.fixes[fi].v1;
      if (slot < 0) break;
      if (!wait_all(sm.raw + fi, i / 4 & 1, sm.abort_flag, 32)) break;
      uint8_t* base = sm.v + slot * L::kTile;
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {
        const int v = half ? v1 : v0;
#pragma unroll 1
        for (int c = lane; c < (64 - v) * (D / 8); c += 32) {
          const int r = v + c / (D / 8), ch = c % (D / 8);
          *reinterpret_cast<uint4*>(base + half * (L::kTile / 2) + (r >> 3) * L::kGroup + (ch >> 3) * 1024 + (r & 7) * 128 +
                                    (ch & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
        }
      }
      fence_proxy_async_smem();  // these stores before the tensor core's reads
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(sm.vfull + slot);
        mbar_arrive(sm.fixdone + fi);
      }
    }
  } else if (warp >= 4) {
    Softmax<D, R, kList> softmax(p, sm, tmem);
    softmax.run();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, L::kTmem);
  }
  if (after_pairs) grid_wait();
}

template <int D, int R>
cudaError_t launch_r(const RowsParams& p, const CUtensorMap& tm_q, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                     int grid, bool after_pairs, cudaStream_t stream) {
  using L = Layout<D, R>;
  auto kern = p.blocks ? few_rows_kernel<D, R, true> : few_rows_kernel<D, R, false>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kAlloc);
  if (e != cudaSuccess) return e;
  return launch_dependent(kern, dim3(grid), 32 * L::kWarps, L::kAlloc, stream, tm_q, tm_k, tm_v, p, after_pairs ? 1 : 0);
}
template <int D>
cudaError_t launch_d(const RowsParams& p, const CUtensorMap& tm_q, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                     int grid, bool after_pairs, cudaStream_t stream) {
  if (p.unit_rows <= 4) return launch_r<D, 4>(p, tm_q, tm_k, tm_v, grid, after_pairs, stream);
  if (p.unit_rows <= 8) return launch_r<D, 8>(p, tm_q, tm_k, tm_v, grid, after_pairs, stream);
  if (p.unit_rows <= 16) return launch_r<D, 16>(p, tm_q, tm_k, tm_v, grid, after_pairs, stream);
  return launch_r<D, kFewRows>(p, tm_q, tm_k, tm_v, grid, after_pairs, stream);
}

}  // namespace

cudaError_t launch_few_rows(const RowsParams& p, const CUtensorMap& tm_q, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                            int grid, bool after_pairs, cudaStream_t stream) {
  return p.d == 64 ? launch_d<64>(p, tm_q, tm_k, tm_v, grid, after_pairs, stream)
                   : launch_d<128>(p, tm_q, tm_k, tm_v, grid, after_pairs, stream);
}

cudaError_t status_word_few_rows(uint32_t** at) { return cudaGetSymbolAddress(reinterpret_cast<void**>(at), g_rows_status); }

}  // namespace attn

// extern "C" boundary of the operators on a paged cache beyond one decode
// step: block tables from request lengths, decode behind a shared prefix, key
// bounds, block selection and attention over selected blocks.  Argument checks
// and dispatch; declared in include/attn.h.
#include <cmath>
#include <cstdint>
#include <cstring>
#include <cuda_runtime.h>

#include "../../include/attn.h"
#include "launch.h"

namespace {

constexpr long long kIntMax = 0x7fffffffLL;
constexpr double kLog2e = 1.4426950408889634;

bool off(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; }

// Memory of n bytes at p; empty where p is NULL.
struct Extent {
  uintptr_t at, end;
};
Extent bytes_at(const void* p, long long n) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(p);
  return {at, p && n > 0 ? at + static_cast<uintptr_t>(n) : at};
}
bool overlap(const Extent& a, const Extent& b) { return a.at < b.end && b.at < a.end; }
// Whether one of the first `outs` overlaps another of the n.
bool outputs_overlap(const Extent* e, int outs, int n) {
  for (int i = 0; i < outs; ++i)
    for (int j = i + 1; j < n; ++j)
      if (overlap(e[i], e[j])) return true;
  return false;
}

// A block table [B, max_blocks] of pages of page_size rows.
attn_status check_table(const int* block_table, int max_blocks, int page_size, int num_pages, const int* seqlens,
                        int B, long long extra) {
  if (B < 1 || max_blocks < 1 || num_pages < 1) return ATTN_ERR_INVALID_ARG;
  if (page_size < 64 || page_size % 64 != 0) return ATTN_ERR_INVALID_ARG;
  if (B > 65535) return ATTN_ERR_UNSUPPORTED;
  if (static_cast<long long>(max_blocks) * page_size + extra + 256 > kIntMax) return ATTN_ERR_UNSUPPORTED;
  if (!block_table || !seqlens) return ATTN_ERR_INVALID_ARG;
  if (off(block_table, 4) || off(seqlens, 4)) return ATTN_ERR_MISALIGNED;
  return ATTN_OK;
}

attn_status check_paging(const int* block_table, int max_blocks, int page_size, int num_pages, const int* seqlens,
                         const int* lens, const int* free_pages, const int* free_count, const int* free_count_out,
                         int B, int Nn) {
  if (Nn < 0) return ATTN_ERR_INVALID_ARG;
  const attn_status st = check_table(block_table, max_blocks, page_size, num_pages, seqlens, B, Nn);
  if (st != ATTN_OK) return st;
  if (!free_pages || !free_count || !free_count_out) return ATTN_ERR_INVALID_ARG;
  if (off(lens, 4) || off(free_pages, 4) || off(free_count, 4) || off(free_count_out, 4)) return ATTN_ERR_MISALIGNED;
  return ATTN_OK;
}

attn_status check_heads(int Nq, int Hq, int Hkv, int d) {
  if (Nq < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0) return ATTN_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
  return ATTN_OK;
}

// Tokens of a launch of the selection: at most 2^26 scores, 65535 tokens (the
// grid's z).
long long select_tokens(int B, int Nq, int Hkv, long long n_blocks) {
  const long long tokens = static_cast<long long>(B) * Nq;
  long long t = (1LL << 26) / (Hkv * n_blocks);
  t = t < 1 ? 1 : (t > 65535 ? 65535 : t);
  return t < tokens ? t : tokens;
}
long long select_tiles(long long n_blocks) { return (n_blocks + 127) / 128; }

// The arguments that both attention calls share.
attn_status check_rows_args(const void* q, const void* k_pages, const void* v_pages, const int* block_table,
                            int max_blocks, int page_size, int num_pages, const int* seqlens, const void* o,
                            const float* lse, int B, int Nq, int Hq, int Hkv, int d, float scale) {
  attn_status st = check_heads(Nq, Hq, Hkv, d);
  if (st == ATTN_OK) st = check_table(block_table, max_blocks, page_size, num_pages, seqlens, B, Nq);
  if (st != ATTN_OK) return st;
  if (!std::isfinite(scale)) return ATTN_ERR_INVALID_ARG;
  if (Hq / Hkv > 128) return ATTN_ERR_UNSUPPORTED;  // a token's heads of a group fit one tile of rows
  if (static_cast<long long>(B) * Nq * Hq > kIntMax - 4096) return ATTN_ERR_UNSUPPORTED;
  if (static_cast<long long>(num_pages) * (page_size / 8) > kIntMax) return ATTN_ERR_UNSUPPORTED;  // coordinates of the pool
  if (!q || !k_pages || !v_pages || !o || !lse) return ATTN_ERR_INVALID_ARG;
  if (off(q, 16) || off(k_pages, 16) || off(v_pages, 16) || off(o, 16) || off(lse, 4)) return ATTN_ERR_MISALIGNED;
  const long long rows = static_cast<long long>(B) * Nq * Hq;
  if (overlap(bytes_at(q, 2 * rows * d), bytes_at(o, 2 * rows * d))) return ATTN_ERR_INVALID_ARG;
  return ATTN_OK;
}

size_t round32(size_t x) { return (x + 31) & ~size_t(31); }
size_t rows_workspace(const attn::RowsSizes& z, int B, int d, bool lists) {
  const size_t rows = static_cast<size_t>(z.pair_rows + z.lane_pieces * z.unit_rows);
  // rows of pieces start at a multiple of 32 bytes, wherever the workspace does
  return 16 + round32(lists ? 0 : (static_cast<size_t>(B) + 3) * sizeof(long long)) + rows * (d + 1) * sizeof(float);
}

// Attention over listed blocks, block by block: its workspace, laid out from a multiple of 32 bytes on.
struct ByBlockSpace {
  size_t o_part, tiles, starts, lse_part, counts, n_tiles, rank, order, end;
};
ByBlockSpace by_block_space(const attn::ByBlockSizes& z, int Hkv, int d, long long n_blocks) {
  ByBlockSpace w;
  w.o_part = 0;
  w.tiles = static_cast<size_t>(z.rows) * d * 4;
  w.starts = w.tiles + static_cast<size_t>(z.groups) * z.tile_cap * 16;
  w.lse_part = w.starts + static_cast<size_t>(z.groups) * Hkv * n_blocks * 8;
  w.counts = w.lse_part + static_cast<size_t>(z.rows) * 4;
  w.n_tiles = w.counts + static_cast<size_t>(z.groups) * Hkv * n_blocks * 4;
  w.rank = w.n_tiles + static_cast<size_t>(z.groups) * 4;
  w.order = w.rank + static_cast<size_t>(z.entries) * 4;
  w.end = w.order + static_cast<size_t>(z.groups) * z.tile_cap * z.tile_tokens * 4;
  return w;
}
size_t lists_workspace(int B, int Nq, int Hq, int Hkv, int d, int n_sel, long long n_blocks) {
  const attn::ByBlockSizes z = attn::by_block_sizes(B, Nq, Hq, Hkv, d, n_sel, n_blocks);
  if (z.chunks > 0) return 16 + by_block_space(z, Hkv, d, n_blocks).end;
  return rows_workspace(attn::rows_sizes(B, Nq, Hq, Hkv, true), B, d, true);
}

// Both attention calls, behind their checks.  blocks: listed ones, or null.
attn_status attend_rows(const void* q, const void* k_pages, const void* v_pages, const int* block_table, int max_blocks,
                        int page_size, int num_pages, const int* seqlens, const int* blocks, int n_sel, int shared_len,
                        void* o, float* lse, int B, int Nq, int Hq, int Hkv, int d, float scale, void* workspace,
                        size_t workspace_bytes, void* stream) {
  const attn::RowsSizes z = attn::rows_sizes(B, Nq, Hq, Hkv, blocks != nullptr);
  const long long n_blocks = static_cast<long long>(max_blocks) * (page_size / 64);
  if (!workspace || off(workspace, 16) ||
      workspace_bytes < (blocks ? lists_workspace(B, Nq, Hq, Hkv, d, n_sel, n_blocks) : rows_workspace(z, B, d, false)))
    return ATTN_ERR_WORKSPACE;
  const float scale_log2 = static_cast<float>(static_cast<double>(scale) * kLog2e);
  char* ws = reinterpret_cast<char*>(round32(reinterpret_cast<uintptr_t>(workspace)));
  CUtensorMap tm_q, tm_qs, tm_k, tm_v;
  if (!attn::make_map_pages(&tm_k, k_pages, num_pages, page_size, Hkv, d) ||
      !attn::make_map_pages(&tm_v, v_pages, num_pages, page_size, Hkv, d))
    return ATTN_ERR_LAUNCH;
  const attn::ByBlockSizes by =
      blocks ? attn::by_block_sizes(B, Nq, Hq, Hkv, d, n_sel, n_blocks) : attn::ByBlockSizes{};
  if (by.chunks > 0) {
    const ByBlockSpace w = by_block_space(by, Hkv, d, n_blocks);
    attn::ByBlockParams p;
    std::memset(&p, 0, sizeof p);
    p.q = q;
    p.block_table = block_table;
    p.seqlens = seqlens;
    p.blocks = blocks;
    p.o = o;
    p.lse = lse;
    p.o_part = reinterpret_cast<float*>(ws + w.o_part);
    p.lse_part = reinterpret_cast<float*>(ws + w.lse_part);
    p.tiles = reinterpret_cast<int4*>(ws + w.tiles);
    p.counts = reinterpret_cast<int*>(ws + w.counts);
    p.starts = reinterpret_cast<int2*>(ws + w.starts);
    p.n_tiles = reinterpret_cast<int*>(ws + w.n_tiles);
    p.rank = reinterpret_cast<int*>(ws + w.rank);
    p.order = reinterpret_cast<int*>(ws + w.order);
    p.max_blocks = max_blocks;
    p.page_size = page_size;
    p.num_pages = num_pages;
    p.n_sel = n_sel;
    p.n_blocks = static_cast<int>(n_blocks);
    p.B = B;
    p.Nq = Nq;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.d = d;
    p.chunks = by.chunks;
    p.chunk_tokens = by.chunk_tokens;
    p.tile_tokens = by.tile_tokens;
    p.tile_cap = by.tile_cap;
    p.scale_log2 = scale_log2;
    p.tile_len = attn::FastDiv(static_cast<uint32_t>(by.tile_tokens));
    CUtensorMap tm_o;
    if (!attn::make_map_pieces(&tm_o, p.o_part, by.rows, d)) return ATTN_ERR_LAUNCH;
    return attn::launch_by_block(p, tm_k, tm_v, tm_o, static_cast<cudaStream_t>(stream)) == cudaSuccess ? ATTN_OK
                                                                                                   : ATTN_ERR_LAUNCH;
  }
  attn::RowsParams p;
  std::memset(&p, 0, sizeof p);
  p.block_table = block_table;
  p.seqlens = seqlens;
  p.blocks = blocks;
  p.o = o;
  p.lse = lse;
  p.max_blocks = max_blocks;
  p.page_size = page_size;
  p.num_pages = num_pages;
  p.shared_len = shared_len;
  p.n_sel = n_sel;
  p.B = B;
  p.Nq = Nq;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.d = d;
  p.scale_log2 = scale_log2;
  p.tile_tokens = z.tile_tokens;
  p.pairs = z.pairs;
  p.own_tokens = z.own_tokens;
  p.own_rt = z.own_rt;
  p.unit_tokens = z.unit_tokens;
  p.unit_rows = z.unit_rows;
  p.pair_rows = z.pair_rows;
  if (!blocks) {
    p.sums = reinterpret_cast<long long*>(ws);
    ws += round32((static_cast<size_t>(B) + 3) * sizeof(long long));
  }
  p.o_part = reinterpret_cast<float*>(ws);
  p.lse_part = p.o_part + static_cast<size_t>(z.pair_rows + z.lane_pieces * z.unit_rows) * d;
  const long long tokens = static_cast<long long>(B) * Nq;
  if (!attn::make_map_group(&tm_q, q, tokens, Hkv, Hq / Hkv, d, z.tile_tokens) ||
      !attn::make_map_group(&tm_qs, q, tokens, Hkv, Hq / Hkv, d, z.unit_tokens))
    return ATTN_ERR_LAUNCH;
  return attn::launch_rows(p, tm_q, tm_qs, tm_k, tm_v, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? ATTN_OK
             : ATTN_ERR_LAUNCH;
}

}  // namespace

extern "C" {

attn_status attn_kvcache_reserve_paged(int* block_table, int max_blocks, int page_size, int num_pages,
                                       const int* seqlens, const int* new_lens, const int* free_pages,
                                       const int* free_count, int* new_lens_out, int* seqlens_out, long long* slots,
                                       int* free_count_out, int B, int Nn, void* stream) {
  const attn_status st = check_paging(block_table, max_blocks, page_size, num_pages, seqlens, new_lens, free_pages,
                                      free_count, free_count_out, B, Nn);
  if (st != ATTN_OK) return st;
  if (!new_lens_out) return ATTN_ERR_INVALID_ARG;
  if (off(new_lens_out, 4) || off(seqlens_out, 4) || off(slots, 8)) return ATTN_ERR_MISALIGNED;
  const Extent e[] = {bytes_at(block_table, 4LL * B * max_blocks), bytes_at(new_lens_out, 4LL * B),
                      bytes_at(seqlens_out, 4LL * B), bytes_at(slots, 8LL * B * Nn), bytes_at(free_count_out, 4),
                      bytes_at(seqlens, 4LL * B), bytes_at(new_lens, 4LL * B), bytes_at(free_pages, 4LL * num_pages),
                      bytes_at(free_count, 4)};
  if (outputs_overlap(e, 5, 9)) return ATTN_ERR_INVALID_ARG;
  attn::PagingParams p;
  std::memset(&p, 0, sizeof p);
  p.seqlens = seqlens;
  p.new_lens = new_lens;
  p.free_count = free_count;
  p.free_pages = free_pages;
  p.block_table = block_table;
  p.seqlens_out = seqlens_out;
  p.new_lens_out = new_lens_out;
  p.free_count_out = free_count_out;
  p.slots = Nn > 0 ? slots : nullptr;
  p.max_blocks = max_blocks;
  p.page_size = page_size;
  p.num_pages = num_pages;
  p.B = B;
  p.Nn = Nn;
  return attn::launch_reserve(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? ATTN_OK : ATTN_ERR_LAUNCH;
}

attn_status attn_kvcache_release_paged(const int* block_table, int max_blocks, int page_size, int num_pages,
                                       const int* seqlens, const int* keep_lens, int* free_pages,
                                       const int* free_count, int* free_count_out, int B, void* stream) {
  const attn_status st = check_paging(block_table, max_blocks, page_size, num_pages, seqlens, keep_lens, free_pages,
                                      free_count, free_count_out, B, 0);
  if (st != ATTN_OK) return st;
  if (!keep_lens) return ATTN_ERR_INVALID_ARG;
  const Extent e[] = {bytes_at(free_pages, 4LL * num_pages), bytes_at(free_count_out, 4),
                      bytes_at(block_table, 4LL * B * max_blocks), bytes_at(seqlens, 4LL * B),
                      bytes_at(keep_lens, 4LL * B), bytes_at(free_count, 4)};
  if (outputs_overlap(e, 2, 6)) return ATTN_ERR_INVALID_ARG;
  attn::PagingParams p;
  std::memset(&p, 0, sizeof p);
  p.seqlens = seqlens;
  p.new_lens = keep_lens;
  p.free_count = free_count;
  p.free_list = free_pages;
  p.block_table = const_cast<int*>(block_table);
  p.free_count_out = free_count_out;
  p.max_blocks = max_blocks;
  p.page_size = page_size;
  p.num_pages = num_pages;
  p.B = B;
  return attn::launch_release(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? ATTN_OK : ATTN_ERR_LAUNCH;
}

attn_status attn_kvcache_bounds_paged(const void* k_pages, void* k_bounds, const int* block_table, int max_blocks,
                                      int page_size, int num_pages, const int* seqlens, const int* new_lens, int B,
                                      int Nn, int Hkv, int d, void* stream) {
  if (Nn < 0 || Hkv < 1) return ATTN_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
  const attn_status st = check_table(block_table, max_blocks, page_size, num_pages, seqlens, B, Nn);
  if (st != ATTN_OK) return st;
  if (Hkv > (1 << 20)) return ATTN_ERR_UNSUPPORTED;
  const long long slabs = (static_cast<long long>(Hkv) * d + 511) / 512;
  if ((static_cast<long long>(Nn) / 64 + 2) * slabs > kIntMax) return ATTN_ERR_UNSUPPORTED;
  if (!k_pages || !k_bounds) return ATTN_ERR_INVALID_ARG;
  if (off(k_pages, 16) || off(k_bounds, 16) || off(new_lens, 4)) return ATTN_ERR_MISALIGNED;
  const long long row = 2LL * Hkv * d, rows = static_cast<long long>(num_pages) * page_size;
  if (overlap(bytes_at(k_pages, rows * row), bytes_at(k_bounds, rows / 64 * 2 * row))) return ATTN_ERR_INVALID_ARG;
  if (Nn == 0) return ATTN_OK;
  attn::KeyBoundsParams p;
  std::memset(&p, 0, sizeof p);
  p.k_pages = k_pages;
  p.k_bounds = k_bounds;
  p.block_table = block_table;
  p.seqlens = seqlens;
  p.new_lens = new_lens;
  p.max_blocks = max_blocks;
  p.page_size = page_size;
  p.num_pages = num_pages;
  p.B = B;
  p.Nn = Nn;
  p.Hkv = Hkv;
  p.d = d;
  return attn::launch_key_bounds(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? ATTN_OK : ATTN_ERR_LAUNCH;
}

size_t attn_select_blocks_workspace_size(int B, int Nq, int Hkv, int max_seqlen) {
  if (B < 1 || Nq < 1 || Hkv < 1 || max_seqlen < 64) return 0;
  const long long n = max_seqlen / 64;
  return (static_cast<size_t>(select_tokens(B, Nq, Hkv, n)) * Hkv * (n + 1) + static_cast<size_t>(B) * Hkv * select_tiles(n)) *
         sizeof(float);
}

attn_status attn_select_blocks_paged(const void* q, const void* k_bounds, const int* block_table, int max_blocks,
                                     int page_size, int num_pages, const int* seqlens, int* blocks, int B, int Nq,
                                     int Hq, int Hkv, int d, int topk, int sink, int local, void* workspace,
                                     size_t workspace_bytes, void* stream) {
  attn_status st = check_heads(Nq, Hq, Hkv, d);
  if (st == ATTN_OK) st = check_table(block_table, max_blocks, page_size, num_pages, seqlens, B, Nq);
  if (st != ATTN_OK) return st;
  if (topk < 1 || sink < 0 || local < 0 || static_cast<long long>(sink) + local > topk) return ATTN_ERR_INVALID_ARG;
  const long long tokens = static_cast<long long>(B) * Nq;
  if (Hq / Hkv > 128) return ATTN_ERR_UNSUPPORTED;  // a token's heads of a group fit one tile of rows
  if (Hkv > 65535 || tokens > kIntMax || tokens * Hkv > kIntMax) return ATTN_ERR_UNSUPPORTED;
  if (!q || !k_bounds || !blocks) return ATTN_ERR_INVALID_ARG;
  if (off(q, 16) || off(k_bounds, 16) || off(blocks, 4)) return ATTN_ERR_MISALIGNED;
  const long long cap = static_cast<long long>(max_blocks) * page_size;
  const long long n = cap / 64;
  if (!workspace || off(workspace, 16) ||
      workspace_bytes < attn_select_blocks_workspace_size(B, Nq, Hkv, static_cast<int>(cap)))
    return ATTN_ERR_WORKSPACE;
  attn::SelectParams p;
  std::memset(&p, 0, sizeof p);
  p.q = q;
  p.k_bounds = k_bounds;
  p.block_table = block_table;
  p.seqlens = seqlens;
  p.blocks = blocks;
  p.max_blocks = max_blocks;
  p.page_size = page_size;
  p.num_pages = num_pages;
  p.B = B;
  p.Nq = Nq;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.d = d;
  p.topk = topk;
  p.sink = sink;
  p.local = local;
  p.n_blocks = static_cast<int>(n);
  const long long step = select_tokens(B, Nq, Hkv, n);
  p.scores = static_cast<float*>(workspace);
  p.q_norm = p.scores + step * Hkv * n;
  p.m_norm = p.q_norm + step * Hkv;
  for (long long t = 0; t < tokens; t += step) {
    const int m = static_cast<int>(tokens - t < step ? tokens - t : step);
    if (attn::launch_select(p, static_cast<int>(t), m, static_cast<cudaStream_t>(stream)) != cudaSuccess)
      return ATTN_ERR_LAUNCH;
  }
  return ATTN_OK;
}

size_t attn_fwd_blocks_paged_workspace_size(int B, int Nq, int Hq, int Hkv, int d, int n_sel, int max_seqlen) {
  if (B < 1 || check_heads(Nq, Hq, Hkv, d) != ATTN_OK || Hq / Hkv > 128) return 0;
  if (n_sel < 1 || n_sel > attn::kMaxListed || max_seqlen < 64) return 0;
  return lists_workspace(B, Nq, Hq, Hkv, d, n_sel, max_seqlen / 64);
}

attn_status attn_fwd_blocks_paged(const void* q, const void* k_pages, const void* v_pages, const int* block_table,
                                  int max_blocks, int page_size, int num_pages, const int* seqlens, const int* blocks,
                                  int n_sel, void* o, float* lse, int B, int Nq, int Hq, int Hkv, int d, float scale,
                                  void* workspace, size_t workspace_bytes, void* stream) {
  const attn_status st = check_rows_args(q, k_pages, v_pages, block_table, max_blocks, page_size, num_pages, seqlens,
                                         o, lse, B, Nq, Hq, Hkv, d, scale);
  if (st != ATTN_OK) return st;
  if (n_sel < 1 || !blocks) return ATTN_ERR_INVALID_ARG;
  if (n_sel > attn::kMaxListed) return ATTN_ERR_UNSUPPORTED;
  if (off(blocks, 4)) return ATTN_ERR_MISALIGNED;
  return attend_rows(q, k_pages, v_pages, block_table, max_blocks, page_size, num_pages, seqlens, blocks, n_sel, 0, o,
                     lse, B, Nq, Hq, Hkv, d, scale, workspace, workspace_bytes, stream);
}

size_t attn_splitkv_paged_shared_workspace_size(int B, int Nq, int Hq, int Hkv, int d) {
  if (B < 1 || check_heads(Nq, Hq, Hkv, d) != ATTN_OK || Hq / Hkv > 128) return 0;
  return rows_workspace(attn::rows_sizes(B, Nq, Hq, Hkv, false), B, d, false);
}

attn_status attn_fwd_splitkv_paged_shared(const void* q, const void* k_pages, const void* v_pages,
                                          const int* block_table, int max_blocks, int page_size, int num_pages,
                                          const int* seqlens, int shared_len, void* o, float* lse, int B, int Nq,
                                          int Hq, int Hkv, int d, float scale, void* workspace,
                                          size_t workspace_bytes, void* stream) {
  const attn_status st = check_rows_args(q, k_pages, v_pages, block_table, max_blocks, page_size, num_pages, seqlens,
                                         o, lse, B, Nq, Hq, Hkv, d, scale);
  if (st != ATTN_OK) return st;
  if (shared_len < 0 || shared_len % page_size != 0 || shared_len / page_size > max_blocks) return ATTN_ERR_INVALID_ARG;
  return attend_rows(q, k_pages, v_pages, block_table, max_blocks, page_size, num_pages, seqlens, nullptr, 0,
                     shared_len, o, lse, B, Nq, Hq, Hkv, d, scale, workspace, workspace_bytes, stream);
}

}  // extern "C"

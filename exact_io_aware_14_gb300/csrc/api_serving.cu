// extern "C" boundary of the operators around the attention kernels: norms
// and rotation of queries and keys, appending to a paged cache, decode over a
// paged e4m3 cache.  Argument checks and dispatch; declared in include/attn.h.
#include <cmath>
#include <cstdint>
#include <cstring>
#include <cuda_runtime.h>

#include "../../include/attn.h"
#include "launch.h"

namespace {

constexpr long long kIntMax = 0x7fffffffLL;
constexpr double kLog2e = 1.4426950408889634;

bool off16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }
bool off4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; }

// Memory from the first to the last element of a tensor; empty where p is NULL.
struct Extent {
  uintptr_t at, end;
};
Extent bytes_at(const void* p, long long n) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(p);
  return {at, p && n > 0 ? at + static_cast<uintptr_t>(n) : at};
}
// bf16 rows of `width` elements, `stride` (below 2^31) elements apart
Extent rows_at(const void* p, long long rows, long long stride, long long width) {
  return bytes_at(p, rows > 0 ? 2 * ((rows - 1) * stride + width) : 0);
}
bool overlap(const Extent& a, const Extent& b) { return a.at < b.end && b.at < a.end; }

attn_status check_rope(const float* cosv, const float* sinv, int max_pos, int rot_dim, int interleaved, int d) {
  if (rot_dim < 0 || rot_dim > d || interleaved < 0 || interleaved > 1) return ATTN_ERR_INVALID_ARG;
  if (rot_dim == 0) return ATTN_OK;
  if (!cosv || !sinv || max_pos < 1) return ATTN_ERR_INVALID_ARG;
  if (rot_dim % 16 != 0) return ATTN_ERR_UNSUPPORTED;
  if (off16(cosv) || off16(sinv)) return ATTN_ERR_MISALIGNED;
  return ATTN_OK;
}

attn::RopeParams rope_params(const float* cosv, const float* sinv, int max_pos, int rot_dim, int interleaved) {
  return {cosv, sinv, max_pos, rot_dim, interleaved};
}

// One of the two tensors of the norm-and-rotation calls: H heads, rows
// `stride` elements apart.  `read`: whether the call reads x.
attn_status check_rows(const void* x, long long stride, int H, int d, bool read) {
  if (!read) return ATTN_OK;
  if (!x || stride < static_cast<long long>(H) * d) return ATTN_ERR_INVALID_ARG;
  if (stride % 8 != 0 || off16(x)) return ATTN_ERR_MISALIGNED;
  if (stride > kIntMax) return ATTN_ERR_UNSUPPORTED;
  return ATTN_OK;
}

// Sizes shared by the forward and backward norm-and-rotation calls.
attn_status check_qk_sizes(int B, int N, int Hq, int Hkv, int d) {
  if (B < 1 || N < 0 || Hq < 1 || Hkv < 0) return ATTN_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
  const long long tokens = static_cast<long long>(B) * N;
  if (tokens > kIntMax || static_cast<long long>(Hq) + Hkv > (1 << 20)) return ATTN_ERR_UNSUPPORTED;
  // rows are counted in 31 bits, with room for the numbers past the last
  if (tokens * (static_cast<long long>(Hq) + Hkv) > kIntMax - (1 << 20)) return ATTN_ERR_UNSUPPORTED;
  return ATTN_OK;
}

attn_status check_append(const void* k, long long k_stride, const void* v, long long v_stride, const void* k_pages,
                         const void* v_pages, const int* block_table, int max_blocks, int page_size, int num_pages,
                         const int* seqlens, const int* new_lens, const int* seqlens_out, int B, int Nn, int Hkv,
                         int d) {
  if (B < 1 || Nn < 0 || Hkv < 1 || max_blocks < 1 || num_pages < 1) return ATTN_ERR_INVALID_ARG;
  if (page_size < 64 || page_size % 64 != 0) return ATTN_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
  if (B > 65535 || Hkv > (1 << 20)) return ATTN_ERR_UNSUPPORTED;
  const long long cap = static_cast<long long>(max_blocks) * page_size;
  if (cap + Nn + page_size > kIntMax) return ATTN_ERR_UNSUPPORTED;
  if ((static_cast<long long>(Nn) / page_size + 2) * Hkv > kIntMax) return ATTN_ERR_UNSUPPORTED;
  if (static_cast<long long>(Nn) * Hkv * (d / 16) > kIntMax * 256) return ATTN_ERR_UNSUPPORTED;
  if (!seqlens || !block_table || !k_pages || !v_pages) return ATTN_ERR_INVALID_ARG;
  if (Nn > 0) {
    attn_status st = check_rows(k, k_stride, Hkv, d, true);
    if (st == ATTN_OK) st = check_rows(v, v_stride, Hkv, d, true);
    if (st != ATTN_OK) return st;
  }
  if (off16(k_pages) || off16(v_pages) || off4(block_table) || off4(seqlens) || (new_lens && off4(new_lens)) ||
      (seqlens_out && off4(seqlens_out)))
    return ATTN_ERR_MISALIGNED;
  const Extent lens_out = bytes_at(seqlens_out, 4LL * B);
  if (overlap(lens_out, bytes_at(seqlens, 4LL * B)) || overlap(lens_out, bytes_at(new_lens, 4LL * B)))
    return ATTN_ERR_INVALID_ARG;
  return ATTN_OK;
}

attn_status append(const void* k, long long k_stride, const void* v, long long v_stride, void* k_pages, void* v_pages,
                   float* k_scales, float* v_scales, const int* block_table, int max_blocks, int page_size,
                   int num_pages, const int* seqlens, const int* new_lens, int* seqlens_out, const float* rope_cos,
                   const float* rope_sin, int max_pos, int rot_dim, int interleaved, int B, int Nn, int Hkv, int d,
                   void* stream) {
  attn_status st = check_append(k, k_stride, v, v_stride, k_pages, v_pages, block_table, max_blocks, page_size,
                                num_pages, seqlens, new_lens, seqlens_out, B, Nn, Hkv, d);
  if (st == ATTN_OK) st = check_rope(rope_cos, rope_sin, max_pos, rot_dim, interleaved, d);
  if (st != ATTN_OK) return st;
  // a page's keys and values would be written over each other
  if (Nn > 0 && (k_pages == v_pages || (k_scales && k_scales == v_scales))) return ATTN_ERR_INVALID_ARG;
  attn::AppendParams p;
  std::memset(&p, 0, sizeof p);
  p.k = k;
  p.v = v;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.k_pages = k_pages;
  p.v_pages = v_pages;
  p.k_scales = k_scales;
  p.v_scales = v_scales;
  p.block_table = block_table;
  p.seqlens = seqlens;
  p.new_lens = new_lens;
  p.seqlens_out = seqlens_out;
  p.rope = rope_params(rope_cos, rope_sin, max_pos, rot_dim, interleaved);
  p.max_blocks = max_blocks;
  p.page_size = page_size;
  p.num_pages = num_pages;
  p.B = B;
  p.Nn = Nn;
  p.Hkv = Hkv;
  p.d = d;
  return attn::launch_append(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? ATTN_OK : ATTN_ERR_LAUNCH;
}

}  // namespace

extern "C" {

attn_status attn_qk_norm_rope(const void* q, long long q_stride, const void* k, long long k_stride,
                              const float* q_weight, const float* k_weight, float eps, const float* rope_cos,
                              const float* rope_sin, int max_pos, int rot_dim, int interleaved, const int* positions,
                              void* q_out, void* k_out, int B, int N, int Hq, int Hkv, int d, void* stream) {
  attn_status st = check_qk_sizes(B, N, Hq, Hkv, d);
  if (st == ATTN_OK) st = check_rope(rope_cos, rope_sin, max_pos, rot_dim, interleaved, d);
  if (st != ATTN_OK) return st;
  if ((q_weight || k_weight) && !(std::isfinite(eps) && eps > 0.f)) return ATTN_ERR_INVALID_ARG;
  if (N == 0) return ATTN_OK;
  st = check_rows(q, q_stride, Hq, d, true);
  if (st == ATTN_OK) st = check_rows(k, k_stride, Hkv, d, Hkv > 0);
  if (st != ATTN_OK) return st;
  if (!q_out || (Hkv > 0 && !k_out)) return ATTN_ERR_INVALID_ARG;
  if (off16(q_out) || (Hkv > 0 && off16(k_out)) || off16(q_weight) || off16(k_weight) || off4(positions))
    return ATTN_ERR_MISALIGNED;
  // over an input only in place, where its rows lie as the output's
  const long long tokens = static_cast<long long>(B) * N, q_width = static_cast<long long>(Hq) * d,
                  k_width = static_cast<long long>(Hkv) * d;
  const bool q_same = q_out == q && q_stride == q_width, k_same = k_out == k && k_stride == k_width;
  const Extent qi = rows_at(q, tokens, q_stride, q_width), ki = rows_at(Hkv ? k : nullptr, tokens, k_stride, k_width),
               qo = rows_at(q_out, tokens, q_width, q_width),
               ko = rows_at(Hkv ? k_out : nullptr, tokens, k_width, k_width);
  if ((!q_same && overlap(qo, qi)) || (!k_same && overlap(ko, ki)) || overlap(qo, ki) || overlap(ko, qi) ||
      overlap(qo, ko))
    return ATTN_ERR_INVALID_ARG;
  attn::QkNormRopeParams p;
  std::memset(&p, 0, sizeof p);
  p.q = q;
  p.k = k;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.q_weight = q_weight;
  p.k_weight = k_weight;
  p.eps = eps;
  p.rope = rope_params(rope_cos, rope_sin, max_pos, rot_dim, interleaved);
  p.positions = positions;
  p.q_out = q_out;
  p.k_out = k_out;
  p.B = B;
  p.N = N;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.d = d;
  return attn::launch_qk_norm_rope(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? ATTN_OK : ATTN_ERR_LAUNCH;
}

size_t attn_qk_norm_rope_bwd_workspace_size(int B, int N, int Hq, int Hkv, int d) {
  if (check_qk_sizes(B, N, Hq, Hkv, d) != ATTN_OK) return 0;
  int nbq, nbk;
  attn::qk_norm_rope_bwd_blocks(B, N, Hq, Hkv, d, &nbq, &nbk);
  return static_cast<size_t>(nbq + nbk) * d * sizeof(float);
}

attn_status attn_qk_norm_rope_bwd(const void* dq_out, const void* dk_out, const void* q, long long q_stride,
                                  const void* k, long long k_stride, const float* q_weight, const float* k_weight,
                                  float eps, const float* rope_cos, const float* rope_sin, int max_pos, int rot_dim,
                                  int interleaved, const int* positions, void* dq, void* dk, float* dq_weight,
                                  float* dk_weight, int B, int N, int Hq, int Hkv, int d, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  attn_status st = check_qk_sizes(B, N, Hq, Hkv, d);
  if (st == ATTN_OK) st = check_rope(rope_cos, rope_sin, max_pos, rot_dim, interleaved, d);
  if (st != ATTN_OK) return st;
  const bool norm = q_weight || k_weight;
  if (norm && !(std::isfinite(eps) && eps > 0.f)) return ATTN_ERR_INVALID_ARG;
  if ((q_weight != nullptr) != (dq_weight != nullptr) || (k_weight != nullptr) != (dk_weight != nullptr))
    return ATTN_ERR_INVALID_ARG;
  if (Hkv == 0 && k_weight) return ATTN_ERR_INVALID_ARG;
  if (N == 0 && !norm) return ATTN_OK;
  if (N > 0) {
    st = check_rows(q, q_stride, Hq, d, q_weight != nullptr);
    if (st == ATTN_OK) st = check_rows(k, k_stride, Hkv, d, k_weight != nullptr);
    if (st != ATTN_OK) return st;
    if (!dq_out || !dq || (Hkv > 0 && (!dk_out || !dk))) return ATTN_ERR_INVALID_ARG;
    if (off16(dq_out) || off16(dq) || (Hkv > 0 && (off16(dk_out) || off16(dk)))) return ATTN_ERR_MISALIGNED;
  }
  if (off16(q_weight) || off16(k_weight) || off4(dq_weight) || off4(dk_weight) || off4(positions))
    return ATTN_ERR_MISALIGNED;
  if (norm && (!workspace || off16(workspace) ||
               workspace_bytes < attn_qk_norm_rope_bwd_workspace_size(B, N, Hq, Hkv, d)))
    return ATTN_ERR_WORKSPACE;
  if (N > 0) {
    // over the outputs' gradients only in place, over q and k not at all
    const long long tokens = static_cast<long long>(B) * N, q_width = static_cast<long long>(Hq) * d,
                    k_width = static_cast<long long>(Hkv) * d;
    const Extent qi = rows_at(q_weight ? q : nullptr, tokens, q_stride, q_width),
                 ki = rows_at(k_weight ? k : nullptr, tokens, k_stride, k_width),
                 gq = rows_at(dq_out, tokens, q_width, q_width),
                 gk = rows_at(Hkv ? dk_out : nullptr, tokens, k_width, k_width),
                 dqo = rows_at(dq, tokens, q_width, q_width),
                 dko = rows_at(Hkv ? dk : nullptr, tokens, k_width, k_width);
    if ((dq != dq_out && overlap(dqo, gq)) || (dk != dk_out && overlap(dko, gk)) || overlap(dqo, gk) ||
        overlap(dko, gq) || overlap(dqo, dko) || overlap(dqo, qi) || overlap(dqo, ki) || overlap(dko, qi) ||
        overlap(dko, ki))
      return ATTN_ERR_INVALID_ARG;
  }
  attn::QkNormRopeParams p;
  std::memset(&p, 0, sizeof p);
  p.q = q;
  p.k = k;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.q_weight = q_weight;
  p.k_weight = k_weight;
  p.eps = eps;
  p.rope = rope_params(rope_cos, rope_sin, max_pos, rot_dim, interleaved);
  p.positions = positions;
  p.dq_out = dq_out;
  p.dk_out = dk_out;
  p.dq = dq;
  p.dk = dk;
  p.dq_weight = dq_weight;
  p.dk_weight = dk_weight;
  p.dw_part = static_cast<float*>(workspace);
  p.B = B;
  p.N = N;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.d = d;
  return attn::launch_qk_norm_rope_bwd(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? ATTN_OK
                                                                                             : ATTN_ERR_LAUNCH;
}

attn_status attn_kvcache_append_paged(const void* k, long long k_stride, const void* v, long long v_stride,
                                      void* k_pages, void* v_pages, const int* block_table, int max_blocks,
                                      int page_size, int num_pages, const int* seqlens, const int* new_lens,
                                      int* seqlens_out, const float* rope_cos, const float* rope_sin, int max_pos,
                                      int rot_dim, int interleaved, int B, int Nn, int Hkv, int d, void* stream) {
  return append(k, k_stride, v, v_stride, k_pages, v_pages, nullptr, nullptr, block_table, max_blocks, page_size,
                num_pages, seqlens, new_lens, seqlens_out, rope_cos, rope_sin, max_pos, rot_dim, interleaved, B, Nn,
                Hkv, d, stream);
}

attn_status attn_kvcache_append_paged_fp8(const void* k, long long k_stride, const void* v, long long v_stride,
                                          void* k_pages, void* v_pages, float* k_scales, float* v_scales,
                                          const int* block_table, int max_blocks, int page_size, int num_pages,
                                          const int* seqlens, const int* new_lens, int* seqlens_out,
                                          const float* rope_cos, const float* rope_sin, int max_pos, int rot_dim,
                                          int interleaved, int B, int Nn, int Hkv, int d, void* stream) {
  if (!k_scales || !v_scales) return ATTN_ERR_INVALID_ARG;
  if (off4(k_scales) || off4(v_scales)) return ATTN_ERR_MISALIGNED;
  return append(k, k_stride, v, v_stride, k_pages, v_pages, k_scales, v_scales, block_table, max_blocks, page_size,
                num_pages, seqlens, new_lens, seqlens_out, rope_cos, rope_sin, max_pos, rot_dim, interleaved, B, Nn,
                Hkv, d, stream);
}

// Few sequences: as many splits as a cluster holds, where those are short (one
// of 701 keys, 8 KV heads: 8.0 us by two kernels, 7.1 in a cluster).  Else the
// keys per CTA of the grid, in one or two rounds of equal splits of at most
// 1024 keys; beyond that splits of 1024 (2048 where there are many rounds
// anyway).  Measured on GB300: a serving batch (16 sequences of 1 to 16 K keys,
// 8 KV heads) 56.0 us with splits of 384, 53.7 with 1024; two sequences of 256
// K keys 192, 177 and 172 us with 512, 1024 and 2048.  With a capacity in place of
// the longest length: 701 keys 7.1 us by their length, 8.6 by 4096 and 10.7 by 32 K
// or more; 16384 keys 12.7, 15.2 by 128 K and 20.2 by 1 M; the serving batch 57.5
// and 59.8 by 1 M.
int attn_splitkv_fp8_chunk(int B, int Nq, int Hq, int Hkv, int max_seqlen) {
  if (B < 1 || Nq < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || max_seqlen < 1) return 0;
  const long long rows = static_cast<long long>(Nq) * (Hq / Hkv);
  const long long ctas = rows <= 4 ? 304 : 152;
  const long long blocks = (rows + 15) / 16 < (rows + 23) / 24 ? (rows + 15) / 16 : (rows + 23) / 24;
  const double groups = static_cast<double>(B) * Hkv * blocks;
  for (int splits = 8; splits > 1; splits /= 2) {
    const int chunk = static_cast<int>((static_cast<long long>(max_seqlen) + 64 * splits - 1) / (64 * splits)) * 64;
    if (groups * splits <= ctas && chunk <= 512) return chunk < 128 ? 128 : chunk;
  }
  const double keys = groups * max_seqlen / ctas;
  const double most = keys > 8192 ? 2048 : 1024;
  const double rounds = keys > 2048 ? keys / most : std::ceil(keys / most);
  const double chunk = std::ceil(keys / (rounds < 1 ? 1 : rounds) / 128) * 128;
  return static_cast<int>(chunk < 128 ? 128 : (chunk > most ? most : chunk));
}

attn_status attn_fwd_splitkv_paged_fp8(const void* q, const void* k_pages, const void* v_pages, const float* k_scales,
                                       const float* v_scales, const int* block_table, int max_blocks, int page_size,
                                       int num_pages, const int* seqlens, void* o, float* lse, int B, int Nq, int Hq,
                                       int Hkv, int d, float scale, int chunk, void* workspace, size_t workspace_bytes,
                                       void* stream) {
  if (B < 1 || Nq < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0) return ATTN_ERR_INVALID_ARG;
  if (max_blocks < 1 || num_pages < 1 || page_size < 64 || page_size % 64 != 0) return ATTN_ERR_INVALID_ARG;
  if (chunk < 64 || chunk % 64 != 0 || !std::isfinite(scale)) return ATTN_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
  const long long cap = static_cast<long long>(max_blocks) * page_size;
  if (cap + Nq + 256 > kIntMax || Nq > 64 || B > 65535 || chunk > attn::kMaxChunkFp8 || (cap + chunk - 1) / chunk > 65535 ||
      static_cast<long long>(Nq) * Hq > 65535)
    return ATTN_ERR_UNSUPPORTED;
  // rows, and items (at most one a row and split) with a margin for the numbers past the last, in 31 bits
  if (static_cast<long long>(B) * Nq * Hq * ((cap + chunk - 1) / chunk) > kIntMax - 4096) return ATTN_ERR_UNSUPPORTED;
  if (!q || !k_pages || !v_pages || !k_scales || !v_scales || !block_table || !seqlens || !o || !lse)
    return ATTN_ERR_INVALID_ARG;
  if (off16(q) || off16(k_pages) || off16(v_pages) || off16(o) || off4(k_scales) || off4(v_scales) ||
      off4(block_table) || off4(seqlens) || off4(lse))
    return ATTN_ERR_MISALIGNED;
  const int max_seqlen = static_cast<int>(cap);
  if (!workspace || off16(workspace) ||
      workspace_bytes < attn_splitkv_workspace_size(B, Nq * Hq, max_seqlen, d, chunk))
    return ATTN_ERR_WORKSPACE;
  const long long rows = static_cast<long long>(B) * Nq * Hq;
  if (overlap(bytes_at(q, 2 * rows * d), bytes_at(o, 2 * rows * d))) return ATTN_ERR_INVALID_ARG;
  attn::DecodeFp8Params p;
  std::memset(&p, 0, sizeof p);
  if (!attn::make_map_e4m3(&p.tm_k, k_pages, num_pages, page_size, Hkv, d, 64) ||
      !attn::make_map_e4m3(&p.tm_v, v_pages, num_pages, page_size, Hkv, d, 64))
    return ATTN_ERR_LAUNCH;
  p.q = q;
  p.k_scales = k_scales;
  p.v_scales = v_scales;
  p.block_table = block_table;
  p.seqlens = seqlens;
  p.o = o;
  p.lse = lse;
  p.max_blocks = max_blocks;
  p.page_size = page_size;
  p.num_pages = num_pages;
  p.B = B;
  p.Nq = Nq;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.d = d;
  p.max_seqlen = max_seqlen;
  p.chunk = chunk;
  p.n_split = static_cast<int>((cap + chunk - 1) / chunk);
  const size_t parts = static_cast<size_t>(B) * Nq * Hq * p.n_split;
  p.o_part = static_cast<float*>(workspace);
  p.lse_part = p.o_part + parts * d;
  p.scale_log2 = static_cast<float>(static_cast<double>(scale) * kLog2e);
  return attn::launch_decode_fp8(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? ATTN_OK : ATTN_ERR_LAUNCH;
}

}  // extern "C"

// Host-side interface between the C-ABI layer (api.cu) and the kernel
// translation units.  Internal to the library.
#pragma once
#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/attn.h"
#include "rope.cuh"

namespace attn {

// Device status codes.  Kernels never trap: a wait that runs out of time
// records (site << 8) | code in the unit's status word and the kernel unwinds.
enum DeviceCode : uint32_t { kDevOk = 0, kDevTimeout = 5, kDevBadSeqlen = 6, kDevBadPage = 7,
                             kDevBadPosition = 8 };

// A launch that may start while the kernel before it on the stream ends.  Such
// kernels (grid_depends in ptx.cuh) wait on the device until that kernel is
// done and its writes are visible, before they read or write global memory.
// cluster: blocks of a cluster along x.
template <typename... P, typename... A>
cudaError_t launch_dependent_clusters(void (*kern)(P...), dim3 grid, int cluster, unsigned block, int smem,
                                      cudaStream_t stream, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, P(args)...);
}
template <typename... P, typename... A>
cudaError_t launch_dependent(void (*kern)(P...), dim3 grid, unsigned block, int smem, cudaStream_t stream,
                             const A&... args) {
  return launch_dependent_clusters(kern, grid, 1, block, smem, stream, args...);
}

struct PrefillParams {
  CUtensorMap tm_q, tm_k, tm_v;  // 4-D maps {d, H, N, B}, box {64, 1, 128, 1}, 128-B swizzle
  void* o;
  float* lse;
  int B, Hq, Hkv, Nq, Nk, d;
  int causal;            // 0 none, 1 aligned top-left, 2 aligned bottom-right
  const int* seqlens;    // null, or keys per sequence (cache lengths <= Nk) on the device
  int window_left, window_right;  // local window aligned bottom-right; -1: that side unbounded
  float scale_log2;      // scale * log2(e)
};
cudaError_t launch_prefill(const PrefillParams& p, cudaStream_t stream);

struct DecodeParams {
  CUtensorMap tm_k, tm_v;  // 4-D maps {d, Hkv, max_seqlen, B}, box {64, 1, 64, 1}, 128-B swizzle
  const void* q;
  const int* seqlens;
  void* o;
  float* lse;
  float* o_part;    // [B, Hq, n_split, d]
  float* lse_part;  // [B, Hq, n_split]
  // paged cache (block_table non-null): maps are {d, Hkv, page_size, num_pages}
  const int* block_table;  // [B, max_blocks]
  int max_blocks, page_size, num_pages;
  int B, Hq, Hkv, d, max_seqlen, chunk, n_split;
  float scale_log2;
};
cudaError_t launch_decode(const DecodeParams& p, cudaStream_t stream);

// Host checks of the split-KV decode arguments other than the workspace, in
// the order the entry points report them (no CUDA call).  block_table is
// null for a contiguous cache.
attn_status check_splitkv_args(const void* q, const void* k, const void* v, const int* seqlens, int max_seqlen,
                               const int* block_table, int page_size, const void* o, const float* lse, int B, int Hq,
                               int Hkv, int d, float scale, int chunk);

// Map of an e4m3 page pool {d, Hkv, page_size, num_pages}: box {d, 1, rows, 1}
// of bytes, swizzle as wide as a head row (64 or 128 bytes).  False on failure.
bool make_map_e4m3(CUtensorMap* m, const void* base, int num_pages, int page_size, int Hkv, int d, int box_rows);

// Division of n < 2^31 by a fixed d in [1, 2^31): with 2^s >= d, m = floor(2^32
// (2^s - d) / d) + 1, n / d = (hi(n m) + n) >> s
// (Granlund and Montgomery, "Division by invariant integers using
// multiplication", 1994).
struct FastDiv {
  uint32_t d, m, s;
  FastDiv() = default;
  explicit FastDiv(uint32_t divisor) : d(divisor), s(0) {
    while ((1ull << s) < d) ++s;
    m = static_cast<uint32_t>(((1ull << 32) * ((1ull << s) - d)) / d + 1);
  }
  __host__ __device__ uint32_t div(uint32_t n) const {
    return (static_cast<uint32_t>((static_cast<uint64_t>(n) * m) >> 32) + n) >> s;
  }
};

// Norms and rotation of queries and keys.  Token rows of q and k are q_stride
// and k_stride elements apart; outputs and gradients are dense.
struct QkNormRopeParams {
  const void* q;
  const void* k;
  long long q_stride, k_stride;
  const float* q_weight;  // null: no norm
  const float* k_weight;
  float eps;
  RopeParams rope;
  const int* positions;  // [B, N], or null: 0 .. N-1
  void* q_out;           // forward
  void* k_out;
  const void* dq_out;    // backward
  const void* dk_out;
  void* dq;
  void* dk;
  float* dq_weight;
  float* dk_weight;
  float* dw_part;  // [blocks, d] partial sums
  int B, N, Hq, Hkv, d;
};
cudaError_t launch_qk_norm_rope(const QkNormRopeParams& p, cudaStream_t stream);
cudaError_t launch_qk_norm_rope_bwd(const QkNormRopeParams& p, cudaStream_t stream);
// Blocks of the backward kernel that walk q's rows and k's rows.
void qk_norm_rope_bwd_blocks(int B, int N, int Hq, int Hkv, int d, int* nbq, int* nbk);

// Appending to a paged cache; bf16 pages, or e4m3 pages with scales.
struct AppendParams {
  const void* k;
  const void* v;
  long long k_stride, v_stride;
  void* k_pages;
  void* v_pages;
  float* k_scales;  // null: bf16 pages
  float* v_scales;
  const int* block_table;
  const int* seqlens;
  const int* new_lens;  // null: Nn each
  int* seqlens_out;     // null: not wanted
  RopeParams rope;
  int max_blocks, page_size, num_pages;
  int B, Nn, Hkv, d;
};
cudaError_t launch_append(const AppendParams& p, cudaStream_t stream);

// Split-KV decode over a paged e4m3 cache.
constexpr int kMaxChunkFp8 = 2048;  // keys per split at most
struct DecodeFp8CombineParams {
  const float* o_part;
  const float* lse_part;
  const int* seqlens;
  void* o;
  float* lse;
  int Nq, Hq, max_seqlen, chunk, n_split;
};
struct DecodeFp8Params {
  CUtensorMap tm_k, tm_v;
  const void* q;
  const float* k_scales;
  const float* v_scales;
  const int* block_table;
  const int* seqlens;
  void* o;
  float* lse;
  float* o_part;    // [B, Nq, Hq, n_split, d]
  float* lse_part;  // [B, Nq, Hq, n_split]
  int max_blocks, page_size, num_pages;
  int B, Nq, Hq, Hkv, d, max_seqlen, chunk, n_split;
  float scale_log2;
  // set at launch: query rows of a KV head, its blocks of rows, those of all
  // KV heads, heads of a group, page size, split length
  int rows;
  FastDiv n_rblk, H, G, page, split;
  int cluster;  // CTAs of a cluster, one a split (0: no clusters)
};
cudaError_t launch_decode_fp8(const DecodeFp8Params& p, cudaStream_t stream);

// Device status words, one a kernel unit, of the current device.
cudaError_t status_word_prefill(uint32_t** at);
cudaError_t status_word_decode(uint32_t** at);
cudaError_t status_word_selftest(uint32_t** at);
cudaError_t status_word_rope(uint32_t** at);
cudaError_t status_word_append(uint32_t** at);
cudaError_t status_word_decode_fp8(uint32_t** at);
constexpr int kStatusUnits = 6;
struct StatusWords {
  uint32_t* at[kStatusUnits];
};
// Takes and clears them all on the stream, one round trip, and synchronises it:
// the first that is not 0, in the order given, or 0.
cudaError_t fetch_status(const StatusWords& words, cudaStream_t stream, uint32_t* out);
cudaError_t launch_selftest_wait_timeout(uint64_t limit_ns, cudaStream_t stream);
cudaError_t launch_selftest_exp2_poly(const float* x, float* y, long long n, cudaStream_t stream);
cudaError_t launch_read_probe(const void* buf, long long n16, unsigned long long* sink, cudaStream_t stream);

}  // namespace attn

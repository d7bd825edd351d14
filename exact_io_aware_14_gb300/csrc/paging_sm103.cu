// Block tables and slot maps of a paged cache, kept on the GPU: pages for new
// tokens from a free list, and back to it, for sm_103a.
//
// The free list is a stack: free_pages[0 .. count - 1] are free, the last one
// is taken first.  With L tokens in the cache, n new ones and pages of P rows,
// a sequence wants need = ceil((L + n) / P) - ceil(L / P) pages; with the sum
// of the needs before it (base) it takes entries count - 1 - base - j,
// j = 0 .. need - 1, if base + need <= count.  A release counts from the last
// sequence's last page, so it puts back what the same reserve took, in place.
//
// Bound by latency: a few bytes for each sequence, 8 for each slot (256 sequences
// of one new token: 3.2 us a call; 48 prompts of up to 8191 4 us).  So one
// launch, in which every block forms the sums before its sequences again (B
// lengths from L2) in place of a second launch or of waiting for a block; the
// count goes to memory of its own, as blocks that start late still read the
// old one.
#include <cuda_runtime.h>

#include "launch.h"
#include "ptx.cuh"

namespace attn {
namespace {

__device__ uint32_t g_paging_status;

__device__ __forceinline__ void record(uint32_t site, uint32_t code) {
  atomicCAS(&g_paging_status, 0u, (site << 8) | code);
}

constexpr int kThreads = 256;

__device__ __forceinline__ long long block_sum(long long x, long long* s) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = x;
  __syncthreads();
  x = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) x += s[w];
  return x;
}

__device__ __forceinline__ int pages_of(long long tokens, int page_size) {
  return static_cast<int>((tokens + page_size - 1) / page_size);
}

__device__ __forceinline__ int free_count_of(const PagingParams& p, bool report) {
  const int c = *p.free_count;
  if (report && (c < 0 || c > p.num_pages)) record(1, kDevBadPage);
  return min(max(c, 0), p.num_pages);
}

// What sequence b holds and wants: `first` pages before the call, `need` new
// ones, n new tokens (0 where the lengths are out of range or do not fit).
struct Want {
  int len, n, first, need;
};
__device__ __forceinline__ Want want_of(const PagingParams& p, int b, bool report) {
  const long long cap = static_cast<long long>(p.max_blocks) * p.page_size;
  Want w;
  w.len = p.seqlens[b];
  w.n = p.new_lens ? p.new_lens[b] : p.Nn;
  const bool bad = w.len < 0 || w.n < 0 || w.n > p.Nn || w.len + static_cast<long long>(w.n) > cap;
  if (bad) {
    if (report) record(2, kDevBadSeqlen);
    w.len = static_cast<int>(min(max(static_cast<long long>(w.len), 0ll), cap));
    w.n = 0;
  }
  w.first = pages_of(w.len, p.page_size);
  w.need = bad ? 0 : pages_of(static_cast<long long>(w.len) + w.n, p.page_size) - w.first;
  return w;
}

__device__ __forceinline__ int checked_page(const PagingParams& p, int pg) {
  if (pg < 0 || pg >= p.num_pages) record(3, kDevBadPage);
  return pg;
}

// Block (x, y): the sequences of range y; of their slots the x-th part, with
// x = 0 the tables and lengths too.
__global__ void __launch_bounds__(kThreads) reserve_kernel(const PagingParams p) {
  grid_depends();
  __shared__ long long s_sum[kThreads / 32];
  const int b0 = static_cast<int>(static_cast<long long>(blockIdx.y) * p.B / gridDim.y);
  const int b1 = static_cast<int>((blockIdx.y + 1ll) * p.B / gridDim.y);
  const bool lead = blockIdx.x == 0;
  const int count = free_count_of(p, lead && b0 == 0 && threadIdx.x == 0);
  long long base = 0;
  for (int b = threadIdx.x; b < b0; b += kThreads) base += want_of(p, b, false).need;
  base = block_sum(base, s_sum);
  for (int b = b0; b < b1; ++b) {
    const Want w = want_of(p, b, lead && threadIdx.x == 0);
    const bool served = w.need == 0 || base + w.need <= count;
    const int granted = served ? w.n : 0;
    int* row = p.block_table + static_cast<long long>(b) * p.max_blocks;
    // page of block `blk` of this sequence's new tokens
    const int* top = p.free_pages + (count - 1 - base + w.first);
    if (lead) {
      if (served)
        for (int j = threadIdx.x; j < w.need; j += kThreads) row[w.first + j] = checked_page(p, top[-(w.first + j)]);
      if (threadIdx.x == 0) {
        p.new_lens_out[b] = granted;
        if (p.seqlens_out) p.seqlens_out[b] = w.len + granted;
        // the one sequence at which the list runs short, or the last one
        if (w.need > 0 && base <= count && base + w.need > count)
          *p.free_count_out = static_cast<int>(count - base);
        else if (b == p.B - 1 && base + w.need <= count)
          *p.free_count_out = static_cast<int>(count - base - w.need);
      }
    }
    if (p.slots) {
      long long* out = p.slots + static_cast<long long>(b) * p.Nn;
      for (long long i = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x; i < p.Nn;
           i += static_cast<long long>(gridDim.x) * kThreads) {
        long long slot = -1;
        if (i < granted) {
          const int pos = w.len + static_cast<int>(i), blk = pos / p.page_size;
          const int pg = checked_page(p, blk < w.first ? row[blk] : top[-blk]);
          if (pg >= 0 && pg < p.num_pages) slot = static_cast<long long>(pg) * p.page_size + pos % p.page_size;
        }
        out[i] = slot;
      }
    }
    base += w.need;
  }
}

// Pages that sequence b gives back: blocks keep .. keep + n - 1.
__device__ __forceinline__ int2 back_of(const PagingParams& p, int b, bool report) {
  const long long cap = static_cast<long long>(p.max_blocks) * p.page_size;
  const int len = p.seqlens[b], keep = p.new_lens[b];
  if (keep < 0 || keep > len || len > cap) {
    if (report) record(4, kDevBadSeqlen);
    return make_int2(0, 0);
  }
  const int first = pages_of(keep, p.page_size);
  return make_int2(first, pages_of(len, p.page_size) - first);
}

__global__ void __launch_bounds__(kThreads) release_kernel(const PagingParams p) {
  grid_depends();
  __shared__ long long s_sum[kThreads / 32];
  // sequences are numbered from the last one here
  const int r0 = static_cast<int>(static_cast<long long>(blockIdx.y) * p.B / gridDim.y);
  const int r1 = static_cast<int>((blockIdx.y + 1ll) * p.B / gridDim.y);
  const int count = free_count_of(p, r0 == 0 && threadIdx.x == 0);
  long long base = 0;
  for (int r = threadIdx.x; r < r0; r += kThreads) base += back_of(p, p.B - 1 - r, false).y;
  base = count + block_sum(base, s_sum);
  for (int r = r0; r < r1; ++r) {
    const int b = p.B - 1 - r;
    const int2 w = back_of(p, b, threadIdx.x == 0);
    const int* row = p.block_table + static_cast<long long>(b) * p.max_blocks + w.x;
    for (int j = threadIdx.x; j < w.y; j += kThreads) {
      const long long at = base + (w.y - 1 - j);
      if (at < p.num_pages)
        p.free_list[at] = checked_page(p, row[j]);
      else
        record(5, kDevBadPage);  // more pages than there are
    }
    base += w.y;
    if (r == p.B - 1 && threadIdx.x == 0)
      *p.free_count_out = static_cast<int>(min(base, static_cast<long long>(p.num_pages)));
  }
}

}  // namespace

cudaError_t launch_reserve(const PagingParams& p, cudaStream_t stream) {
  const unsigned y = static_cast<unsigned>(p.B < 1024 ? p.B : 1024);
  // slots: up to 2048 for each block where there are many
  unsigned x = p.slots ? static_cast<unsigned>((static_cast<long long>(p.Nn) + 2047) / 2048) : 1u;
  if (x < 1u) x = 1u;
  if (x > 64u) x = 64u;
  return launch_dependent(reserve_kernel, dim3(x, y), kThreads, 0, stream, p);
}

cudaError_t launch_release(const PagingParams& p, cudaStream_t stream) {
  const unsigned y = static_cast<unsigned>(p.B < 1024 ? p.B : 1024);
  return launch_dependent(release_kernel, dim3(1, y), kThreads, 0, stream, p);
}

cudaError_t status_word_paging(uint32_t** at) { return cudaGetSymbolAddress(reinterpret_cast<void**>(at), g_paging_status); }

}  // namespace attn

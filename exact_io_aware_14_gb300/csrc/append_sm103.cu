// Appending keys and values of new tokens to a paged cache, keys rotated to
// their position on the way, for sm_103a: a bf16 cache, or e4m3 codes with
// one scale for each page and KV head.
//
// New row i of sequence b goes to position pos = seqlens[b] + i, that is row
// pos % page_size of page block_table[b][pos / page_size].
//
// 8-bit form.  value = code * scale, the scale a power of two: the smallest
// s with amax <= 448.5 s (448 is e4m3's largest value and 448.5 rounds to
// it), amax the largest magnitude that the page's rows of this head hold, at
// least 2^-100.  A power of two makes the division by it exact, so a new
// value is rounded once, and an older code whose page's scale is raised is
// divided by a power of two: exact but for codes that fall below e4m3's
// smallest normal value.  A page that starts with this call (its row 0 is
// new) takes its scale from the new rows alone; otherwise it is the larger of
// its scale, taken up to the next power of two where it came from elsewhere
// and is none, and the new rows' scale.
// The scale has to be known before a code is written, so a block keeps its
// rotated values in registers between the two: as bf16 rounded to odd (cut
// off, the last bit set where anything was cut), from which rounding to
// e4m3's four significant bits or fewer gives what rounding the fp32 value
// gives (Boldo and Melquiond, "Emulation of a FMA and correctly rounded sums:
// proved algorithms using rounding to odd", 2008: two spare bits are enough).
//
// Both are bound by memory: one read of the new rows, one write of the cache
// rows; single tokens by latency.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "launch.h"
#include "ptx.cuh"
#include "rope.cuh"

namespace attn {
namespace {

__device__ uint32_t g_append_status;

__device__ __forceinline__ void record(uint32_t site, uint32_t code) {
  atomicCAS(&g_append_status, 0u, (site << 8) | code);
}

// Cache length before the call and new rows of sequence b, clamped to what
// the cache holds.
struct Span {
  int len, n;
};
__device__ __forceinline__ Span span_of(const AppendParams& p, int b, bool report) {
  const long long cap = static_cast<long long>(p.max_blocks) * p.page_size;
  int len = p.seqlens[b], n = p.new_lens ? p.new_lens[b] : p.Nn;
  const bool bad = len < 0 || len > cap || n < 0 || n > p.Nn;
  len = len < 0 ? 0 : (len > cap ? static_cast<int>(cap) : len);
  n = n < 0 ? 0 : (n > p.Nn ? p.Nn : n);
  const bool full = len + static_cast<long long>(n) > cap;
  if (full) n = static_cast<int>(cap - len);
  if (report && (bad || full)) record(1, kDevBadSeqlen);
  return {len, n};
}

// Page of block blk of sequence b, or -1 (recorded; nothing is written there).
__device__ __forceinline__ int page_of(const AppendParams& p, int b, int blk) {
  const int pg = p.block_table[static_cast<long long>(b) * p.max_blocks + blk];
  if (pg < 0 || pg >= p.num_pages) {
    record(2, kDevBadPage);
    return -1;
  }
  return pg;
}

__device__ __forceinline__ int checked_pos(int pos, int max_pos) {
  if (pos >= max_pos) {
    record(3, kDevBadPosition);
    return max_pos - 1;
  }
  return pos;
}

// ---------------------------------------------------------------------------
// bf16 cache: D/16 threads hold one head's K and V row; kHeads heads of a
// token share its cosines and sines.
constexpr int kThreads = 256;

template <int D, int kHeads, bool kInter>
__global__ void __launch_bounds__(kThreads) append_bf16_kernel(const AppendParams p, int per) {
  grid_depends();
  constexpr int kTPR = D / 16;
  const int l = threadIdx.x % kTPR;
  const int b = blockIdx.y;
  const long long i = (static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x) / kTPR;
  const Span s = span_of(p, b, blockIdx.x == 0 && threadIdx.x == 0);
  if (p.seqlens_out && blockIdx.x == 0 && threadIdx.x == 0) p.seqlens_out[b] = s.len + s.n;
  const int row = static_cast<int>(i / per);
  const int h0 = static_cast<int>(i % per) * kHeads;
  if (row >= s.n) return;
  const int nh = min(kHeads, p.Hkv - h0);
  const long long token = static_cast<long long>(b) * p.Nn + row;
  const __nv_bfloat16* k = static_cast<const __nv_bfloat16*>(p.k) + token * p.k_stride + static_cast<long long>(h0) * D;
  const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(p.v) + token * p.v_stride + static_cast<long long>(h0) * D;
  const int2 ch = row_chunks(l, p.rope.rot);
  uint4 rk[kHeads][2], rv[kHeads][2];
#pragma unroll
  for (int h = 0; h < kHeads; ++h) {
    if (h < nh) {
      rk[h][0] = *reinterpret_cast<const uint4*>(k + h * D + 8 * ch.x);
      rk[h][1] = *reinterpret_cast<const uint4*>(k + h * D + 8 * ch.y);
      rv[h][0] = *reinterpret_cast<const uint4*>(v + h * D + 8 * ch.x);
      rv[h][1] = *reinterpret_cast<const uint4*>(v + h * D + 8 * ch.y);
    }
  }
  const int pos = s.len + row;
  const int pg = page_of(p, b, pos / p.page_size);
  Angles ang;
  if (p.rope.rot > 0) load_angles(p.rope, checked_pos(pos, p.rope.max_pos), l, ang);
  if (pg < 0) return;
  const long long dst = ((static_cast<long long>(pg) * p.page_size + pos % p.page_size) * p.Hkv + h0) * D;
  __nv_bfloat16* ko = static_cast<__nv_bfloat16*>(p.k_pages) + dst;
  __nv_bfloat16* vo = static_cast<__nv_bfloat16*>(p.v_pages) + dst;
#pragma unroll
  for (int h = 0; h < kHeads; ++h) {
    if (h >= nh) break;
    if (p.rope.rot > 0 && l < (p.rope.rot >> 4)) {
      float x[16];
      unpack8(rk[h][0], x);
      unpack8(rk[h][1], x + 8);
      rotate16<kInter, false>(x, ang);
      rk[h][0] = pack8(x);
      rk[h][1] = pack8(x + 8);
    }
    *reinterpret_cast<uint4*>(ko + h * D + 8 * ch.x) = rk[h][0];
    *reinterpret_cast<uint4*>(ko + h * D + 8 * ch.y) = rk[h][1];
    *reinterpret_cast<uint4*>(vo + h * D + 8 * ch.x) = rv[h][0];
    *reinterpret_cast<uint4*>(vo + h * D + 8 * ch.y) = rv[h][1];
  }
}

// ---------------------------------------------------------------------------
// e4m3 cache.  One block per (touched page, KV head, K or V, sequence): it
// alone writes that page's codes and scale of the head, so no two blocks meet.

// Exponent of the scale for largest magnitude amax (finite): amax <= 448.5 *
// 2^e, 448.5 = 0x1.c08p8.
__device__ __forceinline__ int scale_exp(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x604000u ? 1 : 0);
  return max(e, -100);
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// The smallest power of two that is no less than x (0 stays 0; below 2^127).
__device__ __forceinline__ float pow2_up(float x) {
  return __uint_as_float((__float_as_uint(x) + 0x7fffffu) & 0x7f800000u);
}

// Two floats -> two e4m3 codes (nearest, ties to even), `lo` in the low byte;
// NaN stays NaN.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two bf16 of a word rounded to odd from two floats.
__device__ __forceinline__ uint32_t pack_odd(float lo, float hi) {
  const uint32_t a = __float_as_uint(lo), b = __float_as_uint(hi);
  // upper halves; 1 for each lower half that is not 0
  return __byte_perm(a, b, 0x7632) | __vminu2(__byte_perm(a, b, 0x5410), 0x00010001u);
}
// Eight values (four words of bf16) times inv (twice, as bf16: exact, a power
// of two, but where the result is far below e4m3's smallest) -> eight codes.
__device__ __forceinline__ uint32_t e4m3x2_of(uint32_t w, uint32_t inv2) {
  uint32_t t;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(t) : "r"(w), "r"(inv2));
  return e4m3x2(bf16lo(t), bf16hi(t));
}
__device__ __forceinline__ uint2 e4m3x8(const uint4& u, uint32_t inv2) {
  return make_uint2(e4m3x2_of(u.x, inv2) | (e4m3x2_of(u.y, inv2) << 16),
                    e4m3x2_of(u.z, inv2) | (e4m3x2_of(u.w, inv2) << 16));
}
// The word with every infinity made NaN (e4m3 has none, and saturating would hide them).
__device__ __forceinline__ uint32_t inf_to_nan(uint32_t w) {
  if ((w & 0x7fffu) == 0x7f80u) w |= 0x40u;
  if ((w & 0x7fff0000u) == 0x7f800000u) w |= 0x400000u;
  return w;
}
// Largest magnitudes of the words' low and high halves (NaN left out), as bf16 pairs.
__device__ __forceinline__ uint32_t max_abs_pair(uint32_t w, uint32_t m) {
  asm("{\n\t.reg .b32 t;\n\tabs.bf16x2 t, %1;\n\tmax.bf16x2 %0, %0, t;\n\t}" : "+r"(m) : "r"(w));
  return m;
}
__device__ __forceinline__ float max_abs8(const uint4& u, float m) {
  const uint32_t p = max_abs_pair(u.w, max_abs_pair(u.z, max_abs_pair(u.y, max_abs_pair(u.x, 0u))));
  return fmax3(m, bf16lo(p), bf16hi(p));
}
// One e4m3 pair -> two floats (through f16, which holds every e4m3 value).
__device__ __forceinline__ float2 from_e4m3x2(uint16_t u) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(u));
  float lo, hi;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(lo), "=f"(hi)
      : "r"(h));
  return make_float2(lo, hi);
}
// Four codes times f (at most 1, a power of two but for a scale that was none), rounded again.
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float f) {
  const float2 a = from_e4m3x2(static_cast<uint16_t>(w & 0xffffu)), b = from_e4m3x2(static_cast<uint16_t>(w >> 16));
  return e4m3x2(a.x * f, a.y * f) | (e4m3x2(b.x * f, b.y * f) << 16);
}

// kKeep: rows a thread keeps at most (the page has no more than kBlock * 16 /
// D * kKeep new ones); 0: any number, read and rotated a second time for the
// codes.  Four rows a thread and 64 registers (60 to 64 bytes of them spilled),
// so that an SM holds 1024 threads, in the smallest blocks that hold a page's
// rows.  Measured on 49 K
// new tokens, 8 heads, d = 128, pages of 64 / 128 / 256 rows: blocks of 128
// threads 61 us / - / -, 256 threads 84 / 68 / -, 512 threads 144 / 97 / 74;
// 256 threads with eight rows and 128 registers 124 / 91 / 75; rows read twice
// 109 at 256; clusters of 128-thread blocks that exchange their largest values
// - / 79 / 83.  Pages that the largest block does not hold are read twice: 512 and
// 1024 rows of d = 128 105 and 120 us, 1024 rows of d = 64 53 (512 rows, kept: 38).
template <int D, int kBlock, int kKeep, bool kInter>
__global__ void __launch_bounds__(kBlock, 1024 / kBlock) append_e4m3_kernel(const AppendParams p) {
  grid_depends();
  constexpr int kTPR = D / 16;
  constexpr int kRows = kBlock / kTPR;  // rows a round of the block covers
  const int b = blockIdx.y;
  const bool is_v = blockIdx.z != 0;
  const int h = blockIdx.x % p.Hkv, j = blockIdx.x / p.Hkv;
  const bool first = blockIdx.x == 0 && !is_v && threadIdx.x == 0;
  const Span s = span_of(p, b, first);
  if (p.seqlens_out && first) p.seqlens_out[b] = s.len + s.n;
  if (s.n == 0) return;
  const int blk = s.len / p.page_size + j;
  if (blk >= p.max_blocks) return;
  const int start = blk * p.page_size;  // position of the page's row 0
  const int lo = max(s.len, start) - start;
  const int hi = static_cast<int>(min(static_cast<long long>(s.len) + s.n - start, static_cast<long long>(p.page_size)));
  if (hi <= lo) return;  // past the last touched page
  // the page's number is asked for here and looked at behind the rows' loads
  const int pg = p.block_table[static_cast<long long>(b) * p.max_blocks + blk];
  const RopeParams& rope = p.rope;
  const int l = threadIdx.x % kTPR, r0 = threadIdx.x / kTPR;
  const int2 ch = row_chunks(l, rope.rot);
  const bool turn = !is_v && l < (rope.rot >> 4);
  const long long stride = is_v ? p.v_stride : p.k_stride;
  // row r of the page is new row start + r - len of the sequence
  const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(is_v ? p.v : p.k) +
                             (static_cast<long long>(b) * p.Nn + start - s.len) * stride + static_cast<long long>(h) * D;
  auto load_row = [&](int r, uint4 (&u)[2]) {
    const __nv_bfloat16* row = src + r * stride;
    u[0] = *reinterpret_cast<const uint4*>(row + 8 * ch.x);
    u[1] = *reinterpret_cast<const uint4*>(row + 8 * ch.y);
  };
  // Row r as the codes are taken from it (rotated, rounded to odd), its largest
  // magnitude into m: of the fp32 values, as rounding to odd can pass the
  // scale's border.  NaN is left out, with finite_only infinities too (they
  // become NaN).
  auto take_row = [&](int r, uint4 (&u)[2], float& m, bool finite_only) {
    if (turn) {
      Angles ang;
      load_angles(rope, checked_pos(start + r, rope.max_pos), l, ang);
      float x[16];
      unpack8(u[0], x);
      unpack8(u[1], x + 8);
      rotate16<kInter, false>(x, ang);
#pragma unroll
      for (int i = 0; i < 16; i += 2) {
        if (finite_only) {
          if (fabsf(x[i]) == INFINITY) x[i] = NAN;
          if (fabsf(x[i + 1]) == INFINITY) x[i + 1] = NAN;
        }
        m = fmax3(m, fabsf(x[i]), fabsf(x[i + 1]));
      }
      u[0] = make_uint4(pack_odd(x[0], x[1]), pack_odd(x[2], x[3]), pack_odd(x[4], x[5]), pack_odd(x[6], x[7]));
      u[1] = make_uint4(pack_odd(x[8], x[9]), pack_odd(x[10], x[11]), pack_odd(x[12], x[13]), pack_odd(x[14], x[15]));
    } else {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        if (finite_only)
          u[c] = make_uint4(inf_to_nan(u[c].x), inf_to_nan(u[c].y), inf_to_nan(u[c].z), inf_to_nan(u[c].w));
        m = max_abs8(u[c], m);
      }
    }
  };
  constexpr int kHeld = kKeep > 0 ? kKeep : 1;
  uint4 held[kHeld][2];
  auto largest = [&](bool finite_only) {
    float m = 0.f;
    if (kKeep > 0) {
#pragma unroll
      for (int i = 0; i < kHeld; ++i) {
        held[i][0] = held[i][1] = make_uint4(0u, 0u, 0u, 0u);
        if (lo + i * kRows + r0 < hi) load_row(lo + i * kRows + r0, held[i]);
      }
#pragma unroll
      for (int i = 0; i < kHeld; ++i)
        if (lo + i * kRows + r0 < hi) take_row(lo + i * kRows + r0, held[i], m, finite_only);
    } else {
      for (int r = lo + r0; r < hi; r += kRows) {
        uint4 u[2];
        load_row(r, u);
        take_row(r, u, m, finite_only);
      }
    }
    return m;
  };
  __shared__ float s_max[2][kBlock / 32];
  auto block_max = [&](float m, int k) {
    m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));  // m >= 0: ordered as integers
    if ((threadIdx.x & 31) == 0) s_max[k][threadIdx.x >> 5] = m;
    __syncthreads();  // also: every thread has read the old scale before it is written
#pragma unroll
    for (int w = 0; w < kBlock / 32; ++w) m = fmaxf(m, s_max[k][w]);
    return m;
  };
  const float mine = largest(false);
  if (pg < 0 || pg >= p.num_pages) {  // uniform: the rows are dropped
    if (threadIdx.x == 0) record(2, kDevBadPage);
    return;
  }
  const long long pitch = static_cast<long long>(p.Hkv) * D;
  uint8_t* dst = static_cast<uint8_t*>(is_v ? p.v_pages : p.k_pages) + static_cast<long long>(pg) * p.page_size * pitch +
                 static_cast<long long>(h) * D;
  float* scale = (is_v ? p.v_scales : p.k_scales) + static_cast<long long>(pg) * p.Hkv + h;
  const float was = lo > 0 ? *scale : 0.f;

  float amax = block_max(mine, 0);
  const bool inf = amax == INFINITY;  // rare: take the infinities out
  if (inf) amax = block_max(largest(true), 1);
  const float now = fmaxf(pow2_up(was), pow2(scale_exp(amax)));
  const float inv = 1.f / now;  // exact: a power of two
  const uint32_t inv2 = pack_bf16x2(inv, inv);
  if (threadIdx.x == 0) *scale = now;
  if (lo > 0 && now != was) {
    const float f = was * inv;
    for (long long i = threadIdx.x; i < static_cast<long long>(lo) * (D / 16); i += kBlock) {
      uint4* q = reinterpret_cast<uint4*>(dst + i / (D / 16) * pitch + i % (D / 16) * 16);
      uint4 u = *q;
      u.x = rescale4(u.x, f);
      u.y = rescale4(u.y, f);
      u.z = rescale4(u.z, f);
      u.w = rescale4(u.w, f);
      *q = u;
    }
  }
  auto put = [&](int r, const uint4 (&u)[2]) {
    *reinterpret_cast<uint2*>(dst + r * pitch + 8 * ch.x) = e4m3x8(u[0], inv2);
    *reinterpret_cast<uint2*>(dst + r * pitch + 8 * ch.y) = e4m3x8(u[1], inv2);
  };
  if (kKeep > 0) {
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const int r = lo + i * kRows + r0;
      if (r < hi) put(r, held[i]);
    }
  } else {
    for (int r = lo + r0; r < hi; r += kRows) {
      uint4 u[2];
      load_row(r, u);
      float m = 0.f;
      take_row(r, u, m, inf);
      put(r, u);
    }
  }
}

// Two heads a thread group: one, two and four took 5.0, 5.6 and 6.9 us for the
// chunk of five prompts (9 K tokens, 4 heads, d = 64), 3.8, 3.5 and 4.3 for
// 1.5 K tokens of 8 heads of 128, 63.0, 62.9 and 63.6 for 49 K.
constexpr int kHeads = 2;

template <int D>
cudaError_t launch_bf16(const AppendParams& p, cudaStream_t stream) {
  const int per = (p.Hkv + kHeads - 1) / kHeads;
  const long long threads = static_cast<long long>(p.Nn) * per * (D / 16);
  // one block at least: it writes seqlens_out
  const long long blocks = threads > 0 ? (threads + kThreads - 1) / kThreads : 1;
  const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>(p.B));
  return p.rope.inter ? launch_dependent(append_bf16_kernel<D, kHeads, true>, grid, kThreads, 0, stream, p, per)
                      : launch_dependent(append_bf16_kernel<D, kHeads, false>, grid, kThreads, 0, stream, p, per);
}

template <int D, int kBlock, int kKeep>
cudaError_t launch_e4m3_as(const AppendParams& p, dim3 grid, cudaStream_t stream) {
  return p.rope.inter ? launch_dependent(append_e4m3_kernel<D, kBlock, kKeep, true>, grid, kBlock, 0, stream, p)
                      : launch_dependent(append_e4m3_kernel<D, kBlock, kKeep, false>, grid, kBlock, 0, stream, p);
}

template <int D>
cudaError_t launch_e4m3(const AppendParams& p, cudaStream_t stream) {
  const int pages = static_cast<int>((static_cast<long long>(p.Nn) + p.page_size - 2) / p.page_size) + 1;
  const dim3 grid(static_cast<unsigned>(pages) * p.Hkv, static_cast<unsigned>(p.B), 2u);
  const int rows = p.Nn < p.page_size ? p.Nn : p.page_size;  // new rows of a page at most
  // few new rows: the smallest block, for latency (64 sequences' single tokens
  // 2.9 us, with blocks of 256 threads 5.4)
  if (rows <= 64 * 16 / D) return launch_e4m3_as<D, 64, 1>(p, grid, stream);
  if (rows <= 128 * 16 / D * 4) return launch_e4m3_as<D, 128, 4>(p, grid, stream);
  if (rows <= 256 * 16 / D * 4) return launch_e4m3_as<D, 256, 4>(p, grid, stream);
  if (rows <= 512 * 16 / D * 4) return launch_e4m3_as<D, 512, 4>(p, grid, stream);
  return launch_e4m3_as<D, 256, 0>(p, grid, stream);
}

}  // namespace

cudaError_t launch_append(const AppendParams& p, cudaStream_t stream) {
  if (p.k_scales) return p.d == 64 ? launch_e4m3<64>(p, stream) : launch_e4m3<128>(p, stream);
  return p.d == 64 ? launch_bf16<64>(p, stream) : launch_bf16<128>(p, stream);
}

cudaError_t status_word_append(uint32_t** at) { return cudaGetSymbolAddress(reinterpret_cast<void**>(at), g_append_status); }

}  // namespace attn

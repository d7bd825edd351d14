/*
 * attn.h -- C ABI of the GB300 (sm_103a) exact attention forward library
 * (libattn_sm103.so).
 *
 * What is computed.  For query row i of head hq in batch b:
 *     O[b,i,hq,:] = sum_j P_ij V[b,j,hkv,:],   P_ij = exp(s_ij - LSE_i),
 *     s_ij = scale * <Q[b,i,hq,:], K[b,j,hkv,:]>   (-inf where masked),
 *     LSE_i = ln sum_j exp(s_ij),
 * i.e. O = softmax(scale * Q K^T + mask) V plus the per-row natural-log
 * log-sum-exp ("FlashAttention: Part 2", chizkidd.github.io, section 2.1
 * for the function and section 1.3 for the one LSE per row).  The result is
 * reached by tiling over K/V blocks with a running max and sum (same page,
 * section 6.2); the N x N score matrix is never written to memory.
 *
 * Grouped heads: Hkv divides Hq and query head hq reads KV head
 * hq / (Hq / Hkv) (pyshine.com flash-attention tour, "Why You Need This":
 * K and V may carry fewer heads than Q when the counts divide).
 * Masks: causal aligned top-left (key j visible to row i iff j <= i) or
 * bottom-right, and a local window (attn_fwd_window, attn_fwd_kvcache).
 * A row that sees no key gets O = 0 and LSE = -inf.
 *
 * Layout: every tensor is dense and row-major, BSHD with d innermost:
 *     q, o : [B, Nq, Hq, d]  bf16
 *     k, v : [B, Nk, Hkv, d] bf16
 *     lse  : [B, Hq, Nq]     fp32
 * Supported head dims: d = 64 and d = 128.
 *
 * Ownership: every pointer is device memory owned by the caller.  The
 * library allocates nothing and keeps no pointer after a call returns.
 * Every call is asynchronous on the given stream (a cudaStream_t passed as
 * void*, NULL for the legacy default stream); nothing synchronises except
 * attn_get_device_status.
 *
 * Errors: arguments are checked on the host before anything is launched; a
 * failed check returns its code and launches nothing.  No exception crosses
 * this interface.  Problems only the device can see (a pipeline wait that
 * ran out of time, a cache length outside [0, max_seqlen]) are recorded in
 * a library-wide device status word that attn_get_device_status reports.
 * When it reports ATTN_ERR_TIMEOUT, the o and lse of the calls made since
 * the previous status read are undefined (they may hold finite values).
 */
#ifndef ATTN_SM103_H
#define ATTN_SM103_H

#include <stddef.h>

/* Exported symbols of the shared library (everything else is hidden). */
#if defined(__GNUC__)
#define ATTN_API __attribute__((visibility("default")))
#else
#define ATTN_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  ATTN_OK = 0,
  ATTN_ERR_INVALID_ARG = 1,  /* a size, head count, scale or pointer is invalid */
  ATTN_ERR_UNSUPPORTED = 2,  /* valid but not built: d not in {64, 128}, ... */
  ATTN_ERR_MISALIGNED = 3,   /* a pointer is not 16-byte aligned */
  ATTN_ERR_LAUNCH = 4,       /* the CUDA runtime refused a launch or a query */
  ATTN_ERR_TIMEOUT = 5,      /* device: a pipeline wait gave up (reported later) */
  ATTN_ERR_DEVICE_ARG = 6,   /* device: a cache length, page index or position was out of range */
  ATTN_ERR_WORKSPACE = 7     /* workspace missing or smaller than required */
} attn_status;

#define ATTN_CAUSAL_NONE 0
#define ATTN_CAUSAL_TOP_LEFT 1
#define ATTN_CAUSAL_BOTTOM_RIGHT 2

/*
 * Prefill / training-shape forward.
 *   q [B,Nq,Hq,d], k and v [B,Nk,Hkv,d] bf16 in; o [B,Nq,Hq,d] bf16 and
 *   lse [B,Hq,Nq] fp32 out.
 *   causal: ATTN_CAUSAL_NONE (0); ATTN_CAUSAL_TOP_LEFT (1): key j is seen
 *            by row i iff j <= i; ATTN_CAUSAL_BOTTOM_RIGHT (2): iff
 *            j <= i + Nk - Nq, so the last query row sees every key (the
 *            alignment the pyshine.com flash-attention tour names; with
 *            Nq > Nk the first Nq - Nk rows see none: O = 0, LSE = -inf).
 *   scale: finite softmax scale applied to Q K^T (1/sqrt(d) usually).
 * Tiled over 128-row query tiles and 128-key K/V tiles: TMA loads into
 * shared memory, tcgen05 MMAs accumulate S = Q K^T and O += P V in Tensor
 * Memory, the softmax runs on CUDA cores with an online running max/sum
 * ("FlashAttention: Part 2", section 6.2), normalisation is deferred to the
 * end and the O rescale is skipped when a row's max did not move
 * ("Trace FlashAttention's evolution through plain PyTorch code", FA2 and
 * FA4 paragraphs); key tiles wholly above the causal diagonal are skipped.
 * Constraints: B, Hq, Hkv >= 1; Nq >= 0; Nk >= 0; Hq % Hkv == 0;
 * d in {64, 128}; all pointers 16-byte aligned (lse: 4-byte) and non-NULL
 * unless B*Nq == 0.  Nq + Nk must stay below 2^31 - 256.
 */
ATTN_API attn_status attn_fwd(const void* q, const void* k, const void* v, void* o, float* lse,
                     int B, int Hq, int Hkv, int Nq, int Nk, int d,
                     int causal, float scale, void* stream);

/*
 * Local (sliding-window) attention: attn_fwd with a window (window_left,
 * window_right).  Query row i sits at key position pos_i = i + Nk - Nq
 * (aligned bottom-right) and sees key j only if
 *     pos_i - window_left <= j <= pos_i + window_right
 * ("FlashAttention: Part 2", section 3.2: local attention keeps i -> j only
 * for |i - j| <= w; the pyshine.com tour, "From Install to Causal
 * Attention", passes the window as a (left, right) pair next to causal, as
 * in causal with (1023, 0)).  A negative side is unbounded; (-1, -1) is
 * attn_fwd.  The window intersects the causal mask chosen by `causal`;
 * with causal = 0, (w, 0) is bottom-right causal attention over the last
 * w + 1 keys.  Key tiles outside every row's window are never loaded.
 * Arguments, constraints and errors otherwise as for attn_fwd; the inputs
 * must be finite wherever a tile is loaded (keys of [0, Nk) in tiles that
 * some row's window touches).
 */
ATTN_API attn_status attn_fwd_window(const void* q, const void* k, const void* v, void* o, float* lse,
                     int B, int Hq, int Hkv, int Nq, int Nk, int d, int causal,
                     int window_left, int window_right, float scale, void* stream);

/*
 * The same forward against a KV cache with a length per sequence: a block
 * of Nq new query rows (a chunk of a prompt, or several decode tokens)
 * attends to the first seqlens[b] keys of sequence b (pyshine.com
 * flash-attention tour, "Why You Need This": prefill and decode against a
 * KV cache with per-sequence lengths).
 *   q [B,Nq,Hq,d] bf16; k_cache, v_cache [B,max_seqlen,Hkv,d] bf16;
 *   seqlens: device int32 [B], each in [0, max_seqlen]; keys at or past
 *            seqlens[b] are never read into the result, whatever they hold;
 *   o [B,Nq,Hq,d] bf16, lse [B,Hq,Nq] fp32 out;
 *   causal: as for attn_fwd, with Nk = seqlens[b]: ATTN_CAUSAL_BOTTOM_RIGHT
 *            puts query row i at cache position seqlens[b] - Nq + i (the
 *            new rows are the last Nq keys of the cache).
 *   window_left, window_right: a local window as for attn_fwd_window,
 *            positions taken with Nk = seqlens[b]; -1, -1 for none.
 * Constraints and errors are those of attn_fwd; a seqlens entry outside
 * [0, max_seqlen] is clamped and reported as ATTN_ERR_DEVICE_ARG by
 * attn_get_device_status.
 */
ATTN_API attn_status attn_fwd_kvcache(const void* q, const void* k_cache, const void* v_cache,
                             const int* seqlens, int max_seqlen, void* o, float* lse,
                             int B, int Hq, int Hkv, int Nq, int d, int causal,
                             int window_left, int window_right, float scale, void* stream);

/*
 * Bytes of workspace attn_fwd_splitkv needs: fp32 partial outputs and
 * partial LSEs for ceil(max_seqlen / chunk) splits of every (b, hq).
 * Returns 0 for invalid arguments.
 */
ATTN_API size_t attn_splitkv_workspace_size(int B, int Hq, int max_seqlen, int d, int chunk);

/*
 * Query-length-one decode against a KV cache, split over the key axis
 * (pyshine.com flash-attention tour, "Why You Need This": with one query
 * the cache is split across thread blocks and the partial results are
 * combined).
 *   q [B,1,Hq,d] bf16; k_cache, v_cache [B,max_seqlen,Hkv,d] bf16;
 *   seqlens: device int32 [B], valid cache length of each sequence
 *            (keys 0 .. seqlens[b]-1 are attended; nothing at or beyond
 *            seqlens[b] is read into the result, whatever it holds);
 *   o [B,1,Hq,d] bf16 and lse [B,Hq,1] fp32 out;
 *   chunk: keys per split, a positive multiple of 64 (1024 typical);
 *   workspace: device memory of at least
 *            attn_splitkv_workspace_size(B, Hq, max_seqlen, d, chunk) bytes,
 *            16-byte aligned, owned by the caller, contents ignored on entry.
 * Two launches on `stream`: the split kernel writes each split's
 * normalised partial output and LSE to the workspace, the combine kernel
 * merges them.  A seqlens entry outside [0, max_seqlen] is clamped and
 * reported as ATTN_ERR_DEVICE_ARG by attn_get_device_status.
 */
ATTN_API attn_status attn_fwd_splitkv(const void* q, const void* k_cache, const void* v_cache,
                             const int* seqlens, int max_seqlen,
                             void* o, float* lse,
                             int B, int Hq, int Hkv, int d, float scale, int chunk,
                             void* workspace, size_t workspace_bytes, void* stream);

/*
 * The same decode against a paged KV cache (pyshine.com flash-attention
 * tour, "Why You Need This": a paged KV cache for serving).  Key k of
 * sequence b lives in row k % page_size of page block_table[b][k / page_size]
 * of the page pools:
 *   k_pages, v_pages [num_pages, page_size, Hkv, d] bf16, 16-byte aligned;
 *   block_table: device int32 [B, max_blocks], row b lists the pages of
 *            sequence b in key order (entries past its length are not read);
 *   page_size: a positive multiple of 64 (the kernel's key tile), with
 *            chunk / page_size + 2 <= 128 (pages of one split);
 *   seqlens: device int32 [B], each in [0, max_blocks * page_size].
 * The other arguments, the workspace (sized for max_seqlen = max_blocks *
 * page_size) and the results are those of attn_fwd_splitkv.  A page index
 * outside [0, num_pages) is replaced by page 0 for the read and reported as
 * ATTN_ERR_DEVICE_ARG by attn_get_device_status.
 */
ATTN_API attn_status attn_fwd_splitkv_paged(const void* q, const void* k_pages, const void* v_pages,
                                            const int* block_table, int max_blocks, int page_size,
                                            int num_pages, const int* seqlens,
                                            void* o, float* lse,
                                            int B, int Hq, int Hkv, int d, float scale, int chunk,
                                            void* workspace, size_t workspace_bytes, void* stream);

/*
 * Split-KV decode that allocates nothing, for callers that cannot call
 * cudaMalloc or pass a workspace: code running inside a custom allocator or
 * memory-pool callback, under a strict no-allocation policy of an inference
 * server's hot loop, or behind a plain C interface with no device memory of
 * its own to spare.  The paper has no counterpart to this entry point.
 *
 * Same arguments and results as attn_fwd_splitkv, minus the workspace: the
 * partial results go to a fixed scratch array compiled into the library,
 * ATTN_SPLITKV_NOALLOC_MAX_BYTES (8 MiB) in size, which every GPU that loads
 * the library holds until the process exits.  That covers, for example,
 * B=16, Hq=32, d=128, max_seqlen=16384, chunk=1024 (about 4.2 MB).
 *   - Arguments are checked as attn_fwd_splitkv checks them, with the same
 *     codes, before the size check; then it returns ATTN_ERR_WORKSPACE,
 *     launching nothing and making no CUDA call, when
 *     attn_splitkv_workspace_size(B, Hq, max_seqlen, d, chunk) exceeds the
 *     scratch size.
 *   - Calls no cudaMalloc, cudaFree or other allocating routine.
 *   - The first call on a device (with that device current) looks up the
 *     scratch's device address once and keeps it until the process exits;
 *     make that first call before any stream capture.  A device reset
 *     (cudaDeviceReset) after that first call is not supported: the kept
 *     address would no longer be valid.  Returns ATTN_ERR_LAUNCH if the
 *     lookup fails.
 *   - If a split's pipeline wait times out, the combine still reads that
 *     split's scratch rows, which then hold an earlier call's values: o and
 *     lse are undefined whenever attn_get_device_status reports
 *     ATTN_ERR_TIMEOUT.
 *   - Every call on a device shares the one scratch array, which keeps the
 *     last call's contents (nothing needs clearing: each call writes every
 *     partial it reads).  Calls whose kernels may overlap on the GPU (on
 *     different streams with no ordering between them) race on it: order
 *     them on one stream or with events.
 */
#define ATTN_SPLITKV_NOALLOC_MAX_BYTES (8u << 20)
ATTN_API attn_status attn_fwd_splitkv_noalloc(const void* q, const void* k_cache, const void* v_cache,
                                              const int* seqlens, int max_seqlen,
                                              void* o, float* lse,
                                              int B, int Hq, int Hkv, int d, float scale, int chunk,
                                              void* stream);

/* ------------------------------------------------------------------------
 * Operators around the attention kernels.  The pages have no counterpart to
 * these; they are what a program runs before attn_fwd (norms and rotation of
 * q and k) and around a decode step (the new tokens go into the paged cache,
 * which may be held in 8 bits).
 *
 * Position rotation (rope_cos, rope_sin, max_pos, rot_dim, interleaved): the
 * first rot_dim of a head's d values are rotated in pairs, pair i of a token
 * at position t by the angle whose cosine and sine are rope_cos[t][i] and
 * rope_sin[t][i] (device fp32 [max_pos, rot_dim / 2], 16-byte aligned):
 *     (a, b) -> (a cos - b sin, b cos + a sin).
 * interleaved 0 pairs x[i] with x[i + rot_dim/2], 1 pairs x[2i] with
 * x[2i + 1].  rot_dim: a multiple of 16 in [0, d]; 0 is no rotation (the
 * tables may then be NULL).  Products and sums are fp32, each rounded by
 * itself.  A position outside [0, max_pos) is clamped into it and reported
 * as ATTN_ERR_DEVICE_ARG by attn_get_device_status.
 * ------------------------------------------------------------------------ */

/*
 * Norms of queries and keys for each head, with the position rotation in the
 * same pass:  y = R(x * w / sqrt(mean(x^2) + eps)) for every head row x.
 *   q [B,N,Hq,d], k [B,N,Hkv,d] bf16 in, with token rows q_stride and
 *            k_stride elements apart (token t = b*N + n starts at t * stride;
 *            Hq*d and Hkv*d for dense tensors, more for a part of a fused
 *            projection's rows); strides are multiples of 8 below 2^31;
 *   q_weight, k_weight: fp32 [d], 16-byte aligned; NULL leaves that tensor
 *            without a norm (rotation only);
 *   eps: finite and > 0 (not looked at when both weights are NULL);
 *   positions: device int32 [B,N], or NULL for 0 .. N-1 in every sequence;
 *   q_out [B,N,Hq,d], k_out [B,N,Hkv,d] bf16 out, dense.  q_out may be q, and
 *            k_out k, where that input is dense; otherwise they must not
 *            overlap the inputs (from first to last element) or each other.
 * Hkv = 0: q alone (k, k_out NULL).  The statistics are fp32 (squares too: values
 * of a normed row below 2^60), the result is rounded once.  Constraints: B, Hq >= 1; N, Hkv >= 0 (Hkv need not divide
 * Hq); d in {64, 128}; tensors 16-byte aligned; Hq + Hkv at most 2^20 and
 * B * N * (Hq + Hkv) below 2^31 - 2^20.
 */
ATTN_API attn_status attn_qk_norm_rope(const void* q, long long q_stride, const void* k, long long k_stride,
                                       const float* q_weight, const float* k_weight, float eps,
                                       const float* rope_cos, const float* rope_sin, int max_pos, int rot_dim,
                                       int interleaved, const int* positions, void* q_out, void* k_out,
                                       int B, int N, int Hq, int Hkv, int d, void* stream);

/* Bytes of workspace attn_qk_norm_rope_bwd needs; 0 for invalid arguments. */
ATTN_API size_t attn_qk_norm_rope_bwd_workspace_size(int B, int N, int Hq, int Hkv, int d);

/*
 * Gradients of attn_qk_norm_rope.  dq_out, dk_out (bf16, dense) are the
 * gradients of q_out, k_out; q, k and the other arguments are the forward
 * call's (its outputs are not needed: the norms are computed again).
 *   dq [B,N,Hq,d], dk [B,N,Hkv,d] bf16 out, dense; dq may be dq_out, dk dk_out;
 *            otherwise they must not overlap the inputs or each other;
 *   dq_weight, dk_weight: fp32 [d] out (written, not added to), NULL exactly
 *            where the weight is NULL; q (k) may be NULL where its weight is;
 *            Hkv = 0 wants k_weight NULL;
 *   workspace: attn_qk_norm_rope_bwd_workspace_size bytes, 16-byte aligned,
 *            contents ignored; may be NULL when both weights are NULL.  Calls
 *            that may run at once (on other streams, in graphs replayed side
 *            by side) need workspaces of their own.
 * Sums over tokens and heads are fp32 in a fixed order: the same call gives
 * the same bits.  N = 0 writes zero weight gradients.
 */
ATTN_API attn_status attn_qk_norm_rope_bwd(const void* dq_out, const void* dk_out, const void* q, long long q_stride,
                                           const void* k, long long k_stride, const float* q_weight,
                                           const float* k_weight, float eps, const float* rope_cos,
                                           const float* rope_sin, int max_pos, int rot_dim, int interleaved,
                                           const int* positions, void* dq, void* dk, float* dq_weight,
                                           float* dk_weight, int B, int N, int Hq, int Hkv, int d,
                                           void* workspace, size_t workspace_bytes, void* stream);

/*
 * Appends the keys and values of new tokens to a paged cache (the layout of
 * attn_fwd_splitkv_paged), the keys rotated to their position on the way.
 * New row i of sequence b goes to position seqlens[b] + i.
 *   k, v [B,Nn,Hkv,d] bf16, token rows k_stride and v_stride elements apart
 *            (as for attn_qk_norm_rope);
 *   k_pages, v_pages [num_pages, page_size, Hkv, d] bf16, updated in place:
 *            rows other than the new tokens' are left as they are; not the same
 *            memory (nor k_scales and v_scales below);
 *   block_table: device int32 [B, max_blocks]; page_size: a multiple of 64;
 *   seqlens: device int32 [B], the lengths before the call;
 *   new_lens: device int32 [B], how many of the Nn rows of each sequence are
 *            real (the rows behind them are not read); NULL: all Nn;
 *   seqlens_out: device int32 [B], receives the lengths after the call (the
 *            seqlens of a decode that follows); NULL where not wanted; must
 *            not overlap seqlens or new_lens.
 * A length outside [0, max_blocks * page_size], a new_lens entry outside
 * [0, Nn], rows that do not fit the table (they are dropped) and page indices
 * outside [0, num_pages) (nothing is written there) are reported as
 * ATTN_ERR_DEVICE_ARG by attn_get_device_status.  A page that a call writes
 * to belongs to one sequence: where two of them list it, what it holds after
 * the call (in an 8-bit cache its older rows and its scale, too) is undefined.
 */
ATTN_API attn_status attn_kvcache_append_paged(const void* k, long long k_stride, const void* v, long long v_stride,
                                               void* k_pages, void* v_pages, const int* block_table, int max_blocks,
                                               int page_size, int num_pages, const int* seqlens, const int* new_lens,
                                               int* seqlens_out, const float* rope_cos, const float* rope_sin,
                                               int max_pos, int rot_dim, int interleaved, int B, int Nn, int Hkv,
                                               int d, void* stream);

/*
 * The same for a cache held in 8 bits: k_pages, v_pages hold e4m3 codes and
 * k_scales, v_scales [num_pages, Hkv] fp32 one scale for each page and KV
 * head; a value is code * scale.  A scale is a power of two: the smallest s
 * with amax <= 448.5 s, at least 2^-100, where amax is the largest finite
 * magnitude among the page's rows of that head.  A page whose row 0 is new
 * takes its scale from the new rows (whatever page and scale held before); a
 * page that the call continues keeps its scale, or has it raised and its
 * older codes divided by the same power of two and rounded again.  A scale
 * written elsewhere (finite, in [0, 2^127]) is first taken up to the next power
 * of two, at least 2^-100, the older codes multiplied by the quotient and
 * rounded again.  New values
 * are rounded once, to nearest (ties to even), from the fp32 rotated value;
 * infinities and NaN are stored as NaN.
 */
ATTN_API attn_status attn_kvcache_append_paged_fp8(const void* k, long long k_stride, const void* v,
                                                   long long v_stride, void* k_pages, void* v_pages, float* k_scales,
                                                   float* v_scales, const int* block_table, int max_blocks,
                                                   int page_size, int num_pages, const int* seqlens,
                                                   const int* new_lens, int* seqlens_out, const float* rope_cos,
                                                   const float* rope_sin, int max_pos, int rot_dim, int interleaved,
                                                   int B, int Nn, int Hkv, int d, void* stream);

/*
 * A split length (keys per split) that suits attn_fwd_splitkv_paged_fp8 for
 * these sizes, with max_seqlen the longest sequence; 0 for invalid arguments.  It
 * depends on the arguments alone.  Given a table's capacity instead (a program
 * that does not know its lengths, the Python binding by default), splits are as
 * long as sequences that fill the table want them, and shorter sequences spread
 * over fewer SMs.
 */
ATTN_API int attn_splitkv_fp8_chunk(int B, int Nq, int Hq, int Hkv, int max_seqlen);

/*
 * Split-KV decode over a paged cache held in 8 bits (as written by
 * attn_kvcache_append_paged_fp8): key j of sequence b is code * scale with
 * the scale of its page and head, likewise its value.  The last Nq tokens of
 * each sequence are the queries, masked causally among themselves: row i sees
 * keys 0 .. seqlens[b] - Nq + i (Nq = 1: the whole cache).
 *   q [B,Nq,Hq,d] bf16, Nq in [1, 64]; o [B,Nq,Hq,d] bf16 and lse [B,Hq,Nq]
 *            fp32 out; a row that sees no key gets O = 0 and LSE = -inf;
 *            o must not overlap q; scores and sums of weights are fp32, the
 *            weights enter the product with V with nine significant bits;
 *   k_pages, v_pages [num_pages, page_size, Hkv, d] e4m3, 16-byte aligned;
 *   k_scales, v_scales fp32 [num_pages, Hkv], finite and >= 0 (any such value,
 *            not powers of two alone; a page whose value scale is below 2^-100
 *            of the largest in its split adds to o with fewer bits, or nothing);
 *   seqlens: device int32 [B], each in [0, max_blocks * page_size], the new
 *            tokens counted; codes behind a sequence's end reach no result,
 *            whatever they hold;
 *   chunk: keys per split, a multiple of 64 in [64, 2048]
 *            (attn_splitkv_fp8_chunk);
 *   workspace: attn_splitkv_workspace_size(B, Nq * Hq, max_blocks * page_size,
 *            d, chunk) bytes, 16-byte aligned, contents ignored; one for each
 *            call that may run at once, as for attn_qk_norm_rope_bwd.
 * B and Nq * Hq are at most 65535, and B * Nq * Hq times the splits of a sequence
 * stays below 2^31 - 4096.
 * Bad lengths and pages are handled as in attn_fwd_splitkv_paged.
 */
ATTN_API attn_status attn_fwd_splitkv_paged_fp8(const void* q, const void* k_pages, const void* v_pages,
                                                const float* k_scales, const float* v_scales, const int* block_table,
                                                int max_blocks, int page_size, int num_pages, const int* seqlens,
                                                void* o, float* lse, int B, int Nq, int Hq, int Hkv, int d,
                                                float scale, int chunk, void* workspace, size_t workspace_bytes,
                                                void* stream);

/* ------------------------------------------------------------------------
 * Operators on a paged cache beyond one decode step.  The pages have no
 * counterpart to these either.  Where a call takes a block table, lengths and
 * pages, their layouts, limits and the reports of bad ones are those of
 * attn_kvcache_append_paged and attn_fwd_splitkv_paged; B is at most 65535.
 * ------------------------------------------------------------------------ */

/*
 * Block tables and slot maps from request lengths: gives each sequence the
 * pages that its new tokens need, on the GPU, so that a captured step needs no
 * host.  Sequence b holds seqlens[b] tokens in the first
 * ceil(seqlens[b] / page_size) entries of its row and asks for new_lens[b] more.
 *   free_pages: device int32 [num_pages], a stack of free pages, of which
 *            entries 0 .. *free_count - 1 are valid; pages are taken from its
 *            end, sequence by sequence, each one's blocks in order.  A sequence
 *            that needs more pages than are left behind those before it gets
 *            none of its tokens, nor does any later one that needs a page;
 *   block_table: the entries of the new pages are written, no others;
 *   new_lens: device int32 [B], each in [0, Nn], or NULL for Nn each;
 *   new_lens_out: device int32 [B], new_lens[b] where the sequence was served,
 *            else 0 (new_lens of the append that follows);
 *   seqlens_out: device int32 [B], seqlens[b] + new_lens_out[b], or NULL;
 *   slots: device int64 [B, Nn], row number in the pools (page * page_size +
 *            row) of each new token, -1 behind the served ones; or NULL;
 *   free_count_out: device int32 [1], entries that remain valid.
 * No output may overlap another or an input (free_count_out is memory of its
 * own: the next call's free_count).  A length out of range, tokens that do not
 * fit the table (such a sequence gets 0), a free count outside [0, num_pages] and
 * a page outside [0, num_pages) are reported as ATTN_ERR_DEVICE_ARG by
 * attn_get_device_status.
 */
ATTN_API attn_status attn_kvcache_reserve_paged(int* block_table, int max_blocks, int page_size, int num_pages,
                                                const int* seqlens, const int* new_lens, const int* free_pages,
                                                const int* free_count, int* new_lens_out, int* seqlens_out,
                                                long long* slots, int* free_count_out, int B, int Nn, void* stream);

/*
 * Gives pages back to the free list: sequence b keeps the first keep_lens[b]
 * of its seqlens[b] tokens (0 where it is finished, less than seqlens where
 * drafted tokens were rejected, the prefix' length where its first pages are
 * shared), and its pages from block ceil(keep_lens[b] / page_size) on become
 * entries *free_count, ... of free_pages, the last sequence's last page first,
 * so that releasing what a reserve took restores the list.  block_table is left
 * as it is.  A keep_lens outside [0, seqlens[b]] (nothing is released) and pages
 * past num_pages of them (dropped) are reported as ATTN_ERR_DEVICE_ARG.  So is an
 * entry of the table outside [0, num_pages), which goes on the list all the same,
 * in its place: leaving it out would shift what is behind it, so each sequence
 * would have to look through the entries of all those released before it.  The
 * list then has to be built anew; a reserve that takes the entry reports it again.
 */
ATTN_API attn_status attn_kvcache_release_paged(const int* block_table, int max_blocks, int page_size, int num_pages,
                                                const int* seqlens, const int* keep_lens, int* free_pages,
                                                const int* free_count, int* free_count_out, int B, void* stream);

/* Bytes of workspace attn_fwd_splitkv_paged_shared needs; 0 for invalid arguments. */
ATTN_API size_t attn_splitkv_paged_shared_workspace_size(int B, int Nq, int Hq, int Hkv, int d);

/*
 * Decode over a paged bf16 cache where the batch shares a prefix: the first
 * shared_len keys of every sequence lie in the same pages, which are read once
 * for all sequences instead of once for each.  The last Nq tokens of each
 * sequence are the queries, masked causally among themselves: row i sees keys
 * 0 .. seqlens[b] - Nq + i, prefix and own ones alike.
 * (Where fewer than Nq of a sequence's rows are new tokens they are its last rows,
 * not its first as in the append; what the rows ahead of them hold is not looked
 * at by any other row.)
 *   q [B,Nq,Hq,d] bf16, Nq >= 1; o [B,Nq,Hq,d] bf16 and lse [B,Hq,Nq] fp32
 *            out; a row that sees no key gets O = 0 and LSE = -inf; o must not
 *            overlap q;
 *   block_table, seqlens: as for attn_fwd_splitkv_paged, the prefix' pages first
 *            in every row and counted in seqlens (a sequence may be shorter than
 *            the prefix); the prefix is read through row 0 of the table;
 *   shared_len: a multiple of page_size in [0, max_blocks * page_size]; with 0
 *            each sequence is read by itself;
 *   workspace: attn_splitkv_paged_shared_workspace_size bytes, 16-byte aligned,
 *            contents ignored; one for each call that may run at once.
 * The weights enter the product with V rounded to bf16, as in attn_fwd (in
 * attn_fwd_splitkv_paged, for one token and nothing in common, they keep 32 bits).  Keys
 * and values that some row sees must be finite, and values of magnitude 2^80 at
 * most, so that no sum of weighted ones passes fp32's range whatever the scores;
 * behind a sequence's end there may be anything.  Hq / Hkv is at most 128, B * Nq * Hq below 2^31 - 4096.
 */
ATTN_API attn_status attn_fwd_splitkv_paged_shared(const void* q, const void* k_pages, const void* v_pages,
                                                   const int* block_table, int max_blocks, int page_size,
                                                   int num_pages, const int* seqlens, int shared_len, void* o,
                                                   float* lse, int B, int Nq, int Hq, int Hkv, int d, float scale,
                                                   void* workspace, size_t workspace_bytes, void* stream);

/*
 * Sparse attention over blocks of 64 keys, in three calls.  Block j of a
 * sequence is its keys 64 j .. 64 j + 63; new token n of Nq sits at position
 * seqlens[b] - Nq + n and sees the keys up to its own.
 * (Of a sequence with fewer than Nq new tokens they are the last rows of q, as
 * in attn_fwd_splitkv_paged_shared.)
 *
 * (1) Bounds of the keys, kept beside the key pages: k_bounds [num_pages,
 * page_size / 64, Hkv, 2, d] bf16 holds for each block, KV head and channel the
 * smallest (0) and the largest (1) value of the block's keys.  The call forms
 * them anew, from the pages, for the blocks that hold any of the last
 * new_lens[b] of sequence b's seqlens[b] tokens (NULL: the last Nn, or all of a
 * shorter sequence), each over all its keys before the sequence's end.  A NaN
 * key makes its channel's bounds NaN.  k_bounds must not overlap k_pages.  A
 * block that several sequences have in common and that holds new tokens of one of
 * them must lie before the end of each (whole pages of a common prefix do).
 */
ATTN_API attn_status attn_kvcache_bounds_paged(const void* k_pages, void* k_bounds, const int* block_table,
                                               int max_blocks, int page_size, int num_pages, const int* seqlens,
                                               const int* new_lens, int B, int Nn, int Hkv, int d, void* stream);

/*
 * (2) Selection: for each new token and KV head the blocks whose bounds allow
 * the largest scores.
 *     score(j) = max over the group's heads h of
 *                sum_i max(q_hi, 0) * hi_ji + min(q_hi, 0) * lo_ji
 * (no key of block j has a larger <q_h, k>).  Of the blocks that the token sees
 * the first `sink` and the last `local` are taken, then those of the largest
 * score, the lower index first among equals, topk in all (all of them where
 * there are no more).
 *   blocks: device int32 [B, Nq, Hkv, topk] out, ascending, -1 behind the last;
 *   sink, local >= 0, sink + local <= topk; Hq / Hkv is at most 128;
 *   workspace: attn_select_blocks_workspace_size(B, Nq, Hkv, max_blocks *
 *            page_size) bytes, 16-byte aligned, contents ignored; one for each
 *            call that may run at once (a wider table may need a little less:
 *            each width has a size of its own).
 * The order is that of the scores in 64 bits (the products exact, the sums in
 * double precision); a score that is not a number ranks as +inf.
 */
ATTN_API size_t attn_select_blocks_workspace_size(int B, int Nq, int Hkv, int max_seqlen);
ATTN_API attn_status attn_select_blocks_paged(const void* q, const void* k_bounds, const int* block_table,
                                              int max_blocks, int page_size, int num_pages, const int* seqlens,
                                              int* blocks, int B, int Nq, int Hq, int Hkv, int d, int topk, int sink,
                                              int local, void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of workspace attn_fwd_blocks_paged needs with n_sel entries a list and
 * tables of max_seqlen keys (max_blocks * page_size); 0 for invalid arguments.
 * The size follows the form that the sizes choose, so it does not rise with each
 * of them: a narrower table may need far more (2048 tokens of 32 heads, 8 KV
 * heads, d = 128, lists of 32: 1.3 MB with tables of 1 M keys, over 1 GB with
 * 128 K).  A program that keeps one buffer for calls of several sizes takes the
 * largest of their own sizes. */
ATTN_API size_t attn_fwd_blocks_paged_workspace_size(int B, int Nq, int Hq, int Hkv, int d, int n_sel,
                                                     int max_seqlen);

/*
 * (3) Attention of each new token over the keys of its listed blocks that it
 * sees.
 *   blocks: device int32 [B, Nq, Hkv, n_sel], in any order; negative entries
 *            are passed over, as are blocks behind the token's position; a block
 *            listed twice counts twice; n_sel is at most 512; an entry past the table is passed over
 *            and reported as ATTN_ERR_DEVICE_ARG by attn_get_device_status;
 *   workspace: attn_fwd_blocks_paged_workspace_size bytes.  Where the table has
 *            16 list entries or more for each of its blocks (and 16384 for a
 *            sequence and KV heads together, at most 8 heads a group), entries are
 *            sorted by block, and it holds what each gives: 4 (d + 1) bytes a head,
 *            of as many tokens as 1 GB takes.
 * The other arguments, limits and results are those of
 * attn_fwd_splitkv_paged_shared.  Nq may be in the thousands (a prompt, or a
 * chunk of one).  Only keys and values that the row sees enter its result; what
 * lies elsewhere may be anything.
 */
ATTN_API attn_status attn_fwd_blocks_paged(const void* q, const void* k_pages, const void* v_pages,
                                           const int* block_table, int max_blocks, int page_size, int num_pages,
                                           const int* seqlens, const int* blocks, int n_sel, void* o, float* lse,
                                           int B, int Nq, int Hq, int Hkv, int d, float scale, void* workspace,
                                           size_t workspace_bytes, void* stream);

/*
 * Synchronises `stream`, then reads and clears the library's device status
 * word.  Returns ATTN_OK, ATTN_ERR_TIMEOUT, ATTN_ERR_DEVICE_ARG, or
 * ATTN_ERR_LAUNCH if the stream itself reports an error.
 */
ATTN_API attn_status attn_get_device_status(void* stream);

/*
 * Self-test of failure detection.  Every wait of the library's kernels on a
 * pipeline barrier is bounded: when it runs out (2 s) the kernel records
 * ATTN_ERR_TIMEOUT, lets its in-flight copies and tensor-core work finish,
 * frees its Tensor Memory and returns, instead of hanging.  This call
 * launches one small kernel on `stream` whose waits can never be satisfied
 * (barriers that nothing completes): one warp gives up after limit_ns
 * (clamped to [1 us, 2 s]) and the other, with the full limit, must give up
 * as soon as it sees the first one's abort.  Afterwards
 * attn_get_device_status returns ATTN_ERR_TIMEOUT once and the context is
 * usable.  Returns ATTN_OK when the kernel was launched.  The pages have no
 * counterpart to this call; it exists so that the timeout path can be
 * tested without a GPU fault.
 */
ATTN_API attn_status attn_selftest_wait_timeout(unsigned long long limit_ns, void* stream);

/*
 * Self-test of the software exponential: y[i] = 2^x[i] computed the way the
 * prefill kernel computes a fraction of the softmax's exponentials when the
 * library is built with ATTN_EXP2_POLY = K > 0 (every K-th pair of a row's
 * p values), which FA4 does on Blackwell to relieve the MUFU unit
 * ("FlashAttention: Part 2", sections 1.7 and 1.8).  Cody and Waite's range
 * reduction x = n + f, |f| <= 1/2, a degree-3 polynomial for 2^f (largest
 * relative error 1.01e-4 over [-1/2, 1/2]) and n added to the exponent; x is
 * clamped to [-125, 64] first.  Present in every build (the default build's
 * prefill uses the MUFU exponential for every p).
 *   x, y: device float32 arrays of n elements, 4-byte aligned.
 * Returns ATTN_OK once launched on `stream`; ATTN_ERR_INVALID_ARG for n < 0
 * or a NULL pointer (n > 0).
 */
ATTN_API attn_status attn_selftest_exp2_poly(const float* x, float* y, long long n, void* stream);

/*
 * Measurement helper: reads `bytes` of device memory at `buf` once, as a
 * plain stream of 16-byte loads with several in flight per thread over the
 * whole GPU, and XORs a fold of the data into *sink (device memory, 8-byte
 * aligned; its value is meaningless, it only keeps the loads).  Timed on a
 * buffer far larger than L2, it gives the HBM read rate a read-bound kernel
 * (the split-KV decode) is measured against, next to the copy rate.  The
 * pages have no counterpart to this call.
 *   buf: 16-byte aligned, bytes a multiple of 16.
 * Returns ATTN_OK once launched on `stream`.
 */
ATTN_API attn_status attn_probe_read_bandwidth(const void* buf, size_t bytes, unsigned long long* sink,
                                               void* stream);

/* Static, human-readable name of a status code. Never NULL. */
ATTN_API const char* attn_status_string(attn_status s);

#ifdef __cplusplus
}
#endif

#endif /* ATTN_SM103_H */

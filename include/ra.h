/*
 * ra.h -- C ABI of libra: packed causal varlen ring attention with zigzag
 * context-parallel (CP) load balancing, for NVIDIA GB300 (sm_103a).
 *
 * All CP ranks are simulated on one GPU: rank r's shard is the slice
 * [off[r], off[r+1]) of one zigzag-permuted buffer, and a ring step that
 * "receives" rank s's K/V reads that slice in place.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - Layout "THD": a token-major tensor [T, H, d], row-major, d contiguous
 *    (the packed layout of flash_attn_varlen_* named in "Attention Mask for
 *    Packed Sequences (via Attention Bias)", EasyDeL #129).
 *  - cu_seqlens: int32 cumulative document lengths, B+1 entries, cu[0] = 0,
 *    non-decreasing, cu[B] = T.  Documents never attend to each other
 *    (same page, opening request).
 *  - GQA: Hq = G * Hkv; query head h reads KV head floor(h / G).
 *  - LSE: natural-log log-sum-exp of the scaled scores, fp32, layout [Hq, T]
 *    (row h holds all tokens of head h).  A row with no allowed key has
 *    lse = -inf and output 0.
 *  - Device pointers must be 16-byte aligned.  "HOST" marks host arrays.
 *  - Every call is asynchronous on `stream` (a cudaStream_t; NULL = legacy
 *    default stream) unless it says otherwise.  The caller owns and
 *    allocates every device buffer, including the workspace; the library
 *    allocates no device memory.
 *  - Errors: argument checks happen on the host before any launch and
 *    return RA_ERR_INVALID_ARG / RA_ERR_UNSUPPORTED / RA_ERR_WORKSPACE with
 *    nothing launched; a failed launch returns RA_ERR_CUDA.  Device-side
 *    faults the kernels detect themselves (a wait that gave up, an index
 *    out of range) are recorded in a status word read by
 *    ra_get_device_status().  ra_last_error() gives a one-line detail of the
 *    last failure on the calling host thread.
 */
#ifndef RA_H_
#define RA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef int ra_status;
enum {
    RA_OK = 0,
    RA_ERR_INVALID_ARG = 1,   /* bad shape, cu_seqlens, pointer, cp, mode   */
    RA_ERR_UNSUPPORTED = 2,   /* valid but not implemented (dtype, d, align) */
    RA_ERR_CUDA = 3,          /* a CUDA runtime call or launch failed       */
    RA_ERR_WORKSPACE = 4,     /* workspace NULL or smaller than required    */
    RA_ERR_TIMEOUT = 5,       /* a device-side wait gave up (status word)   */
    RA_ERR_DEVICE_BOUNDS = 6  /* a kernel caught an out-of-range index      */
};

enum { RA_ZZ_GLOBAL = 0, RA_ZZ_PER_DOC = 1 };        /* zigzag modes       */
enum { RA_BF16 = 0, RA_FP32 = 1 };                   /* element types      */
enum { RA_SCHED_FUSED = 0, RA_SCHED_STEPWISE = 1, RA_SCHED_ALLGATHER = 2 };  /* CP schedules */

/* ------------------------------------------------------------------------
 * ra_zigzag_plan  (HOST, synchronous, no GPU needed)
 *
 * The zigzag split of ring-attention-pytorch #20 ("Zigzag attention
 * support?", the `extract_local` snippet) and maxtext PR #1133 (review
 * comment on load-balanced reordering): a stream of L tokens is cut into
 * n = 2*cp chunks, chunk c = [floor(c*L/n), floor((c+1)*L/n)), and rank r
 * holds chunks r and n-1-r.  When n does not divide L this balanced split
 * is used (chunks differ by at most one token; some may be empty).
 *   mode RA_ZZ_GLOBAL : the stream is the whole packed batch (T tokens).
 *   mode RA_ZZ_PER_DOC: every document is split on its own ("Question about
 *                       varlen ring attention", MiniMax-01 #6, notes that
 *                       zigzag under packing is the hard case).
 * Local token order is increasing packed index in both modes.
 *
 *   cu_seqlens HOST [B+1]             in
 *   perm       HOST [T]     int32     out: perm[i] = packed index of the
 *                                     token in permuted slot i
 *   off        HOST [cp+1]  int32     out: rank r owns slots [off[r], off[r+1])
 *   cu_local   HOST [cp*(B+1)] int32  out: rank r's local cu_seqlens (entry
 *                                     r*(B+1)+b); zero-length docs allowed
 * ------------------------------------------------------------------------ */
ra_status ra_zigzag_plan(const int32_t *cu_seqlens, int B, int cp, int mode,
                         int32_t *perm, int32_t *off, int32_t *cu_local);

/* ------------------------------------------------------------------------
 * ra_zigzag_permute / ra_zigzag_unpermute  (DEVICE)
 *
 * Applies the reordering the maxtext PR #1133 review says the framework
 * must perform before load-balanced CP attention (and undo afterwards):
 *   permute:    y[i, :] = x[perm[i], :]      for i in [0, T)
 *   unpermute:  x[perm[i], :] = y[i, :]
 * Rows are `row_bytes` bytes (H*d*element size for THD tensors); the copy
 * is bit-exact.  perm is a DEVICE int32 array [T] that must be a
 * permutation of [0, T) (an entry outside [0, T) is skipped and recorded
 * as RA_ERR_DEVICE_BOUNDS).  x and y must not overlap.
 * ------------------------------------------------------------------------ */
ra_status ra_zigzag_permute(const void *x, void *y, const int32_t *perm,
                            int64_t T, int64_t row_bytes, void *stream);
ra_status ra_zigzag_unpermute(const void *y, void *x, const int32_t *perm,
                              int64_t T, int64_t row_bytes, void *stream);

/* ------------------------------------------------------------------------
 * ra_varlen_attn_partial  (DEVICE tensors, HOST segment/position arrays)
 *
 * One ring step's attention: local queries against one KV shard, returning
 * the normalised output and its LSE so that partials can be merged
 * ("[Train] Support custom attention with context parallel", FlagScale
 * PR #910: RingAttention with a swappable forward_impl; this is that
 * step).  Allowed pairs:
 *   (i, j) with seg(i) == seg(j) and (causal == 0 or k_pos[j] <= q_pos[i])
 *          and (window < 0 or k_pos[j] >= q_pos[i] - window),
 * where seg is given by cu_seqlens_q / cu_seqlens_k (segment b of Q pairs
 * with segment b of K, nseg segments each).  window: the sliding window,
 * the number of positions a key may lie behind its query (the window_size
 * argument of the cuDNN flash-attention call in "Add Context Parallelism
 * support to cudnn Flash Attention #1133", maxtext); -1 = no window.
 *   q   DEVICE [Tq, Hq, d]      dtype RA_BF16 or RA_FP32
 *   k,v DEVICE [Tk, Hkv, d]     same dtype
 *   cu_seqlens_q, cu_seqlens_k  HOST [nseg+1]
 *   q_pos HOST [Tq], k_pos HOST [Tk]  int32 positions used by the causal
 *                               test (NULL = the local row index)
 *   out DEVICE [Tq, Hq, d] fp32, lse DEVICE [Hq, Tq] fp32 (written in full)
 *   workspace DEVICE, >= ra_partial_workspace_bytes(...) bytes
 * bf16 with d = 128 and G a power of two <= 16 runs on the tensor cores
 * (tcgen05, fp32 accumulation); other shapes and fp32 run a SIMT fp32 path.
 * Host arrays: every call tiles its segments on the host (O(Tq + Tk) work
 * plus O(query tiles x KV tiles) to classify tile pairs) and copies the
 * tables into the workspace on `stream` from host memory, so a call on a
 * capturing stream is refused with RA_ERR_UNSUPPORTED before any work
 * (the ring calls, which cache their plans, can be captured).
 * ra_partial_workspace_bytes is a bound over every position pattern;
 * ra_partial_table_bytes gives the exact bytes the tables of one call take
 * (HOST, no GPU needed; 0 for invalid arguments) and never exceeds it.
 * ------------------------------------------------------------------------ */
size_t ra_partial_workspace_bytes(int64_t Tq, int64_t Tk, int nseg, int Hq, int Hkv, int d, int dtype);
size_t ra_partial_table_bytes(int64_t Tq, int64_t Tk, int Hq, int Hkv, int d, int dtype,
                              const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_k, int nseg,
                              const int32_t *q_pos, const int32_t *k_pos, int causal, int window);
ra_status ra_varlen_attn_partial(const void *q, const void *k, const void *v, int dtype,
                                 int64_t Tq, int64_t Tk, int Hq, int Hkv, int d,
                                 const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_k, int nseg,
                                 const int32_t *q_pos, const int32_t *k_pos,
                                 int causal, int window, float scale,
                                 float *out, float *lse,
                                 void *workspace, size_t ws_bytes, void *stream);

/* ------------------------------------------------------------------------
 * ra_varlen_attn_partial_dev  (DEVICE tensors and DEVICE segment/position
 * arrays)
 *
 * ra_varlen_attn_partial with cu_seqlens_q, cu_seqlens_k [nseg+1], q_pos
 * [Tq] and k_pos [Tk] (NULL = the local row index) in DEVICE memory, as a
 * ring step holds them: the tile tables are built on the GPU (one small
 * kernel, the host planner's tiling row for row) ahead of the tensor-core
 * kernel, so the call makes no host round trip and can be captured in a
 * CUDA graph.  Same allowed pairs, results and workspace bound
 * (ra_partial_workspace_bytes) as ra_varlen_attn_partial; with the same
 * inputs the results are bit-identical to it.  Tensor-core path only
 * (bf16, d = 128, Hq / Hkv a power of two <= 16; else RA_ERR_UNSUPPORTED).
 * The device arrays are checked on the device: segment boundaries that do
 * not start at 0, decrease, or do not end at Tq / Tk (and, with a window,
 * positions outside [0, 2^30)) are recorded as RA_ERR_DEVICE_BOUNDS in the
 * status word (ra_get_device_status) and leave out / lse unwritten.
 * ------------------------------------------------------------------------ */
ra_status ra_varlen_attn_partial_dev(const void *q, const void *k, const void *v, int dtype,
                                     int64_t Tq, int64_t Tk, int Hq, int Hkv, int d,
                                     const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_k, int nseg,
                                     const int32_t *q_pos, const int32_t *k_pos,
                                     int causal, int window, float scale,
                                     float *out, float *lse,
                                     void *workspace, size_t ws_bytes, void *stream);

/* ------------------------------------------------------------------------
 * ra_varlen_attn_partial_noalloc  (DEVICE tensors, HOST segment/position
 * arrays) -- the pages have no counterpart; this is a library convenience.
 *
 * The same computation, arguments and results as ra_varlen_attn_partial,
 * for callers that cannot allocate device memory: a runtime whose memory
 * pool already owns the GPU, a plugin that is handed only its input and
 * output buffers, or code that must not risk the implicit device
 * synchronisation cudaMalloc / cudaFree can cause.  Instead of a caller
 * workspace it uses a static device array of RA_NOALLOC_SCRATCH_BYTES
 * (8 MiB) that every GPU which loads the library holds until the process
 * exits; this call allocates nothing.
 *  - Size limit: a problem whose ra_partial_workspace_bytes(...) exceeds
 *    RA_NOALLOC_SCRATCH_BYTES is rejected with RA_ERR_WORKSPACE (the detail
 *    in ra_last_error() names both sizes); nothing is launched.
 *  - Set-up: the first call on a device (with that device current) looks up
 *    the array's device address and caches it.  Make that first call before
 *    any stream capture.  `stream` must belong to the current device (a
 *    stream of another device is rejected with RA_ERR_INVALID_ARG).  The
 *    cached address lives as long as the device's context: a
 *    cudaDeviceReset after the first call is not supported.
 *  - Sharing: all calls on a device share the one array, which keeps the
 *    last call's contents.  Each call rewrites every table it reads, so no
 *    state carries over, but calls that overlap on the GPU (different
 *    streams, or host threads) race on the array: serialise them.
 * ------------------------------------------------------------------------ */
#define RA_NOALLOC_SCRATCH_BYTES (8u << 20)
ra_status ra_varlen_attn_partial_noalloc(const void *q, const void *k, const void *v, int dtype,
                                         int64_t Tq, int64_t Tk, int Hq, int Hkv, int d,
                                         const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_k, int nseg,
                                         const int32_t *q_pos, const int32_t *k_pos,
                                         int causal, int window, float scale,
                                         float *out, float *lse, void *stream);

/* ------------------------------------------------------------------------
 * ra_lse_merge  (DEVICE)
 *
 * Merges n_parts partial results of the same queries over disjoint key
 * sets (the step that combines ring partials; the pages name the ring
 * schedule, the merge is its textbook completion):
 *   M = max_p lse_p;  lse = M + log(sum_p exp(lse_p - M));
 *   out = sum_p exp(lse_p - lse) * out_p;   all -inf -> out 0, lse -inf.
 *   outs  HOST array [n_parts] of DEVICE fp32 [Tq, Hq, d] pointers
 *   lses  HOST array [n_parts] of DEVICE fp32 [Hq, Tq] pointers
 *   out   DEVICE [Tq, Hq, d] of out_dtype (RA_BF16 or RA_FP32)
 *   lse_out DEVICE [Hq, Tq] fp32 (may be NULL)
 * 1 <= n_parts <= 64, d a multiple of 4 and <= 256.  out may alias
 * outs[0] when out_dtype is RA_FP32 (each element is read before written).
 * ------------------------------------------------------------------------ */
ra_status ra_lse_merge(int n_parts, const float *const *outs, const float *const *lses,
                       int64_t Tq, int Hq, int d, void *out, int out_dtype, float *lse_out,
                       void *stream);

/* ------------------------------------------------------------------------
 * ra_ring_attn_fwd / ra_ring_attn_bwd  (DEVICE tensors, HOST cu_seqlens)
 *
 * The whole simulated ring: zigzag-permute Q/K/V, run the ring over cp
 * simulated ranks (rank r at step t attends to the K/V of rank
 * s = (r - t) mod cp), merge, and return results in the ORIGINAL token
 * order.
 *   sched RA_SCHED_FUSED    : one launch per direction; the ring steps are
 *                             the order in which each query tile visits KV
 *                             tiles and the merge is the on-chip online
 *                             softmax.  Fully masked tiles are skipped
 *                             (pruning, FlagScale PR #910).
 *   sched RA_SCHED_STEPWISE : one partial launch per ring step into fp32
 *                             buffers, then ra_lse_merge and unpermute
 *                             (backward: fp32 dK/dV accumulated per step).
 *   sched RA_SCHED_ALLGATHER: the all-gather form of context parallelism
 *                             (K/V of every rank gathered, then one pass of
 *                             each rank's zigzag queries over them: the
 *                             Llama 3 scheme discussed in "Zigzag attention
 *                             support?", ring-attention-pytorch issue #20,
 *                             and the Transformer-Engine path of maxtext PR
 *                             #1133).  The gathered K/V are the documents in
 *                             original order, tiled per document, so they
 *                             are read in place and never permuted.  Same
 *                             attention as the ring; only the tiling of
 *                             the key side and the rounding order differ.
 *                             Without tensor-core kernels (fp32, other
 *                             shapes) it runs as RA_SCHED_FUSED.
 * Forward:
 *   q DEVICE [T, Hq, d], k, v DEVICE [T, Hkv, d] (dtype), out DEVICE
 *   [T, Hq, d] (dtype), lse DEVICE [Hq, T] fp32.
 * Backward (from the saved lse, textbook gradient):
 *   out, dout DEVICE [T, Hq, d] (dtype), lse DEVICE [Hq, T];
 *   dq DEVICE [T, Hq, d], dk, dv DEVICE [T, Hkv, d] of grad_dtype
 *   (RA_BF16 or RA_FP32; dK/dV are always accumulated in fp32).
 * scale: softmax scale; pass 1/sqrt(d) for the usual attention (maxtext
 * PR #1133, cudnn_flash_attention diff).  cp >= 1.  window: sliding window
 * as in ra_varlen_attn_partial (-1 = none); positions are the original
 * (unpermuted) token indices, so the zigzag reorder leaves the mask intact.
 * workspace: DEVICE, >= ra_ring_workspace_bytes(...) for the same arguments
 * (the size holds for every causal and window setting: the planner's KV
 * tiling, which the mask selects, only changes the size of its tables and
 * the size covers every tiling).  ra_ring_workspace_bytes counts tiles on
 * the host (well under a millisecond for 32768 tokens) and keeps no state;
 * it returns 0 for invalid arguments.
 * On the tensor-core path (bf16, d = 128) the kernels read every tile whose
 * rows form one position run straight from q, k, v (and dout), and the
 * workspace receives rank-ordered copies of the rows of the other tiles
 * only (those that straddle two zigzag chunks); ra_zigzag_permute gives the
 * whole rank-ordered tensor where a caller needs it.
 * Asynchronous on `stream`.  The backward's fused tensor-core path runs its
 * key-side kernel on a second, library-owned stream forked from and joined
 * back to `stream` through events.  Both calls may be captured into a CUDA
 * graph once an uncaptured call with the same cu_seqlens, cp, zz_mode and
 * heads has run (it makes the page-locked table copy and the second
 * stream); otherwise a captured call returns RA_ERR_UNSUPPORTED.
 * ------------------------------------------------------------------------ */
size_t ra_ring_workspace_bytes(int64_t T, int Hq, int Hkv, int d, int dtype,
                               const int32_t *cu_seqlens, int B, int cp, int zz_mode,
                               int sched, int bwd);
ra_status ra_ring_attn_fwd(const void *q, const void *k, const void *v, int dtype,
                           int64_t T, int Hq, int Hkv, int d,
                           const int32_t *cu_seqlens, int B, int cp, int zz_mode,
                           int causal, int window, float scale, int sched,
                           void *out, float *lse,
                           void *workspace, size_t ws_bytes, void *stream);
/* flags of ra_ring_attn_bwd.
 * RA_BWD_FWD_RESERVE: the workspace is a reserve space left by the
 * preceding ra_ring_attn_fwd on the same stream with the same q, k, v
 * (unmodified), dtype, shapes, cu_seqlens, cp, zz_mode, causal and sched,
 * and nothing has written into it since: the rank-ordered Q, K, V rows and
 * the tile tables it holds are reused instead of rebuilt (they are the
 * forward's saved activations).  The library checks on the host that the
 * last forward on this workspace had the same pointers and plan and
 * ignores the flag otherwise; it cannot see changes to the contents. */
#define RA_BWD_FWD_RESERVE 1
ra_status ra_ring_attn_bwd(const void *q, const void *k, const void *v, int dtype,
                           int64_t T, int Hq, int Hkv, int d,
                           const int32_t *cu_seqlens, int B, int cp, int zz_mode,
                           int causal, int window, float scale, int sched,
                           const void *out, const float *lse, const void *dout,
                           void *dq, void *dk, void *dv, int grad_dtype, int flags,
                           void *workspace, size_t ws_bytes, void *stream);

/* ------------------------------------------------------------------------
 * ra_ring_attn_fwd_masked / ra_ring_attn_bwd_masked  (DEVICE tensors, HOST
 * cu_seqlens and bounds)
 *
 * The ring of ra_ring_attn_fwd / bwd under an interval mask instead of the
 * causal flag and the window: the dynamic, per-token attention masks that
 * "[Train] Support custom attention with context parallel" (FlagScale PR
 * #910, description) adds to context parallelism through flex attention,
 * in the form of one key interval per query token:
 *   query i sees key j  iff  same document  and  key_lo[i] <= j <= key_hi[i]
 * (original token indices).  This holds causal (lo = document start,
 * hi = i), sliding-window, chunked-local, prefix-LM (hi = max(i, end of
 * the prefix)) and bidirectional document masks.
 *   key_lo, key_hi HOST int32 [T]: both non-decreasing inside every
 *                  document (else RA_ERR_INVALID_ARG), values in
 *                  (-2^30, 2^30); a row with no key inside its interval
 *                  gets output 0 and lse -inf.
 * Fully masked tile pairs are skipped and fully visible ones run unmasked:
 * the block map comes from each query tile's bound extremes (the pruning
 * of the same PR).  Everything else is as in ra_ring_attn_fwd / bwd, with
 * these limits: the tensor-core path only (bf16, d = 128, Hq / Hkv a power
 * of two <= 16) and the RA_SCHED_FUSED or RA_SCHED_ALLGATHER schedule
 * (otherwise RA_ERR_UNSUPPORTED).  The plan (and so the workspace size)
 * depends on the bounds: size the workspace with
 * ra_ring_workspace_bytes_masked for the same bounds.
 * ------------------------------------------------------------------------ */
size_t ra_ring_workspace_bytes_masked(int64_t T, int Hq, int Hkv, int d, int dtype,
                                      const int32_t *cu_seqlens, int B, int cp, int zz_mode,
                                      const int32_t *key_lo, const int32_t *key_hi, int sched, int bwd);
ra_status ra_ring_attn_fwd_masked(const void *q, const void *k, const void *v, int dtype,
                                  int64_t T, int Hq, int Hkv, int d,
                                  const int32_t *cu_seqlens, int B, int cp, int zz_mode,
                                  const int32_t *key_lo, const int32_t *key_hi, float scale, int sched,
                                  void *out, float *lse, void *workspace, size_t ws_bytes, void *stream);
ra_status ra_ring_attn_bwd_masked(const void *q, const void *k, const void *v, int dtype,
                                  int64_t T, int Hq, int Hkv, int d,
                                  const int32_t *cu_seqlens, int B, int cp, int zz_mode,
                                  const int32_t *key_lo, const int32_t *key_hi, float scale, int sched,
                                  const void *out, const float *lse, const void *dout,
                                  void *dq, void *dk, void *dv, int grad_dtype, int flags,
                                  void *workspace, size_t ws_bytes, void *stream);

/* ------------------------------------------------------------------------
 * ra_rope_fwd / ra_rope_bwd  (DEVICE tensors, HOST frequency table)
 *
 * Rotary positions of queries and keys ahead of the attention, and the
 * gradient behind its backward.  A head has n_pairs rotated pairs: elements
 * (i, i + n_pairs), or with `adjacent` (2i, 2i + 1); elements from
 * 2 * n_pairs on pass through.  Pair i turns by the angle
 *   phi = pos[axes[i]][t] * inv_freq[i]
 *   forward:  (x, y) -> (x cos phi - y sin phi, x sin phi + y cos phi)
 *   backward: the same with -phi (the transposed rotation).
 * Several axes (time, height, width) give each pair the coordinate that
 * axes[i] names.  The angle is reduced exactly: inv_freq / (2 pi) is kept as
 * a 64-bit binary fraction of a turn, so positions over the whole int32 range
 * keep an angle as exact as a 64-bit product.  Its distance to the nearest
 * quarter turn is rounded to fp32 (2.4e-8 rad at most) ahead of the sine and
 * cosine, which are exact to one unit in the last place.
 *   q  DEVICE [T, Hq, d], k DEVICE [T, Hk, d] (k and k_out NULL: queries only);
 *      rows of H*d contiguous elements, q_stride / k_stride elements apart
 *      (a slice of a packed QKV projection); the same for the outputs.  An
 *      output may be its own input (same pointer and stride); otherwise they
 *      must not overlap.
 *   pos DEVICE int32 [n_axes, T].  1 <= n_axes <= 8.
 *   rope->inv_freq HOST double [n_pairs], rope->axes HOST uint8 [n_pairs]
 *      (NULL = axis 0 for every pair).  1 <= n_pairs, 2 * n_pairs <= d.
 * d a multiple of 4, d <= 256; dtype RA_BF16 or RA_FP32.  Rotation in fp32,
 * one rounding at the end.  Any alignment of the element type; 16-byte
 * aligned rows and pair counts of whole 16-byte vectors take the fast path.
 * Can be captured: the table travels with the launch.
 * ------------------------------------------------------------------------ */
typedef struct ra_rope {
    const double *inv_freq;  /* HOST [n_pairs] */
    const uint8_t *axes;     /* HOST [n_pairs] or NULL */
    int32_t n_pairs, n_axes, adjacent;
} ra_rope;
ra_status ra_rope_fwd(const void *q, const void *k, void *q_out, void *k_out, int dtype, int64_t T, int Hq, int Hk,
                      int d, int64_t q_stride, int64_t k_stride, int64_t q_out_stride, int64_t k_out_stride,
                      const int32_t *pos, const ra_rope *rope, void *stream);
ra_status ra_rope_bwd(const void *dq, const void *dk, void *dq_out, void *dk_out, int dtype, int64_t T, int Hq,
                      int Hk, int d, int64_t dq_stride, int64_t dk_stride, int64_t dq_out_stride,
                      int64_t dk_out_stride, const int32_t *pos, const ra_rope *rope, void *stream);

/* A paged cache of keys and values (DEVICE): page p, row r, head h starts at
 * element p * page_stride + r * token_stride + h * head_stride of k and of v,
 * with d contiguous elements.  The strides hold [pages, rows, heads, d] as
 * well as [pages, heads, rows, d] and caches interleaved with each other. */
typedef struct ra_paged_kv {
    void *k, *v;
    int64_t n_pages, page_stride, token_stride, head_stride;
    int32_t page_size, Hkv, d, dtype;
} ra_paged_kv;

/* ------------------------------------------------------------------------
 * ra_kv_cache_append  (DEVICE tensors and DEVICE segment arrays)
 *
 * Writes the new tokens of B sequences into their pages, keys rotated on the
 * way, and rotates the queries beside them, in one launch.  Token j of the
 * n_b = cu_seqlens[b+1] - cu_seqlens[b] new ones of sequence b gets the row
 * of logical index i = kv_lens[b] - n_b + j (kv_lens counts the new tokens):
 * row i % page_size of page page_table[b][i / page_size].
 *   k, v DEVICE [T, Hkv, d] (rows k_stride / v_stride elements apart)
 *   page_table DEVICE int32 [B, table_width]; cu_seqlens DEVICE int32 [B+1];
 *   kv_lens DEVICE int32 [B]
 *   q, q_out DEVICE [T, Hq, d] or both NULL; q_out may be q
 *   pos, rope as in ra_rope_fwd (pos DEVICE int32 [n_axes, T]); rope NULL: nothing is rotated
 *      (q and q_out must then be NULL)
 * cu_seqlens starts at 0 and does not decrease.  Tokens at or behind
 * cu_seqlens[B] (a padded batch) are left alone: neither their q_out rows nor
 * any cache row is written for them.  A token whose logical index or page lies
 * outside the table or the cache is not written and RA_ERR_DEVICE_BOUNDS is
 * recorded (its q_out row is still written).  Two tokens of one call must not
 * name the same cache row (distinct sequences' tables must not share the pages
 * that they append to); which of them a row then holds is not defined, vector
 * by vector.  Capturable; lengths and tables may change between replays.
 * An empty batch (T = 0, also with B = 0) does nothing.
 * Limits on d, dtype and n_pairs as in ra_rope_fwd.
 * ------------------------------------------------------------------------ */
ra_status ra_kv_cache_append(const void *k, const void *v, int64_t k_stride, int64_t v_stride, int64_t T,
                             const ra_paged_kv *cache, const int32_t *page_table, int64_t table_width,
                             const int32_t *cu_seqlens, const int32_t *kv_lens, int B,
                             const void *q, void *q_out, int Hq, int64_t q_stride, int64_t q_out_stride,
                             const int32_t *pos, const ra_rope *rope, void *stream);

/* ------------------------------------------------------------------------
 * ra_paged_attn_fwd  (DEVICE tensors and DEVICE segment arrays)
 *
 * Attention of a batch's new tokens over a paged cache, where sequences may
 * share a prefix whose keys are read for all of them together: once for every
 * 256 query rows (tokens of the group times Hq / Hkv) in bf16 with d 128,
 * Hq / Hkv a power of two up to 128, pages of 8, 16, 32, 64 or a multiple of 128
 * tokens, a positive scale and keys enough (see max_q_len); once for every 64
 * rows in other shapes of bf16 with d 64 or 128; once for every 64, of few keys
 * 16, in fp32 and with other d, in fp32 arithmetic.  Sequence b has
 * n_b = cu_seqlens_q[b+1] - cu_seqlens_q[b] query tokens, the last n_b of its
 * kv_lens[b] cached tokens.  Token j sees
 *   - the whole prefix of its sequence's group, and
 *   - its own sequence's cached keys with logical index
 *     < kv_lens[b] - n_b + j + 1 (causal), or < kv_lens[b] (causal == 0).
 * Groups: sequences prefix_groups[g] .. prefix_groups[g+1] - 1 share the
 * prefix_lens[g] tokens in the pages prefix_table[g] (a sequence outside
 * every group has none; n_groups = 0: no prefix at all).  The prefix's pages
 * are pages of the same cache.
 *   q DEVICE [T, Hq, d] (rows q_stride elements apart), dtype of the cache
 *   out DEVICE [T, Hq, d] contiguous, out_dtype RA_FP32 or the cache's dtype;
 *   lse DEVICE fp32 [Hq, T]: with fp32 the pair is a partial for ra_lse_merge
 *   page_table [B, table_width], prefix_table [n_groups, prefix_width],
 *   cu_seqlens_q [B+1], kv_lens [B], prefix_lens [n_groups],
 *   prefix_groups [n_groups+1]: DEVICE int32
 *   max_q_len: the most query tokens a sequence is expected to have; it and
 *      the tables' widths only choose the kernels (<= 0: not known), results
 *      hold for any n_b
 *   workspace DEVICE, 256-byte aligned, >= ra_paged_attn_workspace_bytes(...);
 *      what it holds ahead of the call does not change the results (bytes that
 *      the call has not written may be read, and are dropped).  Calls in
 *      flight at the same time, and captured graphs that may run so, need
 *      workspaces of their own.
 * Scores, softmax statistics and sums are fp32.  In bf16 with d 64 or 128 and
 * more than 16 query rows a KV head (max_q_len, or T where it is not known and
 * for prefixes, times Hq / Hkv) the weights are rounded to bf16 ahead of their
 * product with V, as in ra_ring_attn_fwd; else they keep 15 bits or more.
 * An empty batch (T = 0, also with B = 0) does nothing.
 * A row without any visible key has output 0 and lse -inf.  Rows at or behind
 * cu_seqlens_q[B] (a padded batch) are not written.  Cache rows at or behind
 * a sequence's length may hold anything (NaN included); a key that some
 * query tokens of a sequence see and others do not must be finite.
 * The device arrays are checked on the device: boundaries that decrease or
 * leave [0, T], groups that decrease or leave [0, B], and lengths outside
 * [0, width * page_size] or above 2^30 are recorded as RA_ERR_DEVICE_BOUNDS
 * and leave out and lse unwritten; a page index outside [0, n_pages) is
 * recorded too, reads nothing, and leaves the rows that meet it unspecified.
 * A NaN in a query or in a key makes the rows that it reaches NaN, lse too.
 * Capturable; the arrays' contents may change between replays.  Deterministic:
 * the same arguments on the same kind of device give the same bits.  Other
 * lengths, table widths, max_q_len, page sizes, strides or signs of the scale
 * may be other kernels and another order of the sums, so the same keys behind a
 * wider table can differ by rounding.  d a multiple
 * of 32, d <= 256; q, out and the cache 16-byte aligned with strides of whole
 * 16 bytes; T * Hq <= 2^30.  out may be q.
 * ------------------------------------------------------------------------ */
size_t ra_paged_attn_workspace_bytes(int64_t T, int B, int n_groups, int Hq, int Hkv, int d, int dtype,
                                     int max_q_len);
ra_status ra_paged_attn_fwd(const void *q, int64_t q_stride, int64_t T, int Hq, const ra_paged_kv *cache,
                            const int32_t *page_table, int64_t table_width, const int32_t *cu_seqlens_q,
                            const int32_t *kv_lens, int B, const int32_t *prefix_table, int64_t prefix_width,
                            const int32_t *prefix_lens, const int32_t *prefix_groups, int n_groups, int causal,
                            int max_q_len, float scale, void *out, int out_dtype, float *lse,
                            void *workspace, size_t ws_bytes, void *stream);

/* Weights of the cache's keys (DEVICE, fp32): page p, row r, head h at w +
 * p * page_stride + r * token_stride + h * head_stride, for the pages, rows
 * and heads of a ra_paged_kv.  They are written, so no two share memory: a
 * stride of 0 (of more than one page, row or head) is refused. */
typedef struct ra_paged_weights {
    float *w;
    int64_t page_stride, token_stride, head_stride;
} ra_paged_weights;

/* ------------------------------------------------------------------------
 * ra_paged_attn_key_weights  (DEVICE tensors and DEVICE segment arrays)
 *
 * The attention weight that each cached key gathers from a batch's new tokens,
 * added to `weights`: what ra_kv_cache_evict goes by.  With q, cache, tables,
 * lengths, groups, causal and scale of a ra_paged_attn_fwd call and the lse
 * that it wrote, for every key of KV head h that sequence b's tokens see,
 *   w += sum over the tokens t that see it and the query heads of h
 *        of exp(scale q.k - lse[head][t]),
 * its own keys and the prefix of its group (for all of the group's sequences
 * together).  A new key's weight is to be 0 ahead of its first call: pages
 * begin with 0, and ra_kv_cache_evict leaves 0 behind what it keeps in place.
 * Query rows that are left out (a call with a part of the rows: cu_seqlens_q,
 * q and lse of those) add nothing, so the weights of the last tokens alone can
 * be gathered as well.  cache->v is not used.
 *   lse DEVICE fp32 [Hq, T]; a row with lse = -inf saw nothing and adds nothing
 * Each weight is added to once, by one thread, and in a fixed order: the same
 * call gives the same bits.  Two sequences (or groups) of one call must not
 * name the same page; keys that sequences share belong into a prefix.
 * Sums are fp32; the products are fp32 in fp32, exact products summed in fp32
 * in bf16.  Cache rows at or behind a sequence's length may hold anything, and
 * their weights are not touched; a NaN in a key makes its own weight NaN, one in
 * a query the weights of all keys that it sees.  Device arrays are checked as
 * in ra_paged_attn_fwd: a bad boundary or length is recorded as
 * RA_ERR_DEVICE_BOUNDS and nothing is added; keys on a page outside the cache
 * are recorded and add nothing.  max_q_len is a hint, as there.  Limits on
 * shapes, alignment and strides as there.  Capturable; no workspace.  An empty
 * batch (T = 0) does nothing.
 * ------------------------------------------------------------------------ */
ra_status ra_paged_attn_key_weights(const void *q, int64_t q_stride, int64_t T, int Hq, const ra_paged_kv *cache,
                                    const ra_paged_weights *weights, const int32_t *page_table, int64_t table_width,
                                    const int32_t *cu_seqlens_q, const int32_t *kv_lens, int B,
                                    const int32_t *prefix_table, int64_t prefix_width, const int32_t *prefix_lens,
                                    const int32_t *prefix_groups, int n_groups, int causal, int max_q_len, float scale,
                                    const float *lse, void *stream);

/* ------------------------------------------------------------------------
 * ra_kv_cache_evict  (DEVICE tensors and DEVICE segment arrays)
 *
 * Holds B cached sequences to a budget.  Of the n = kv_lens[b] keys of a
 * sequence with more than keep_b stay the first `sinks`, the last `recent` and,
 * of those between, the ones of the largest weight (ties: the lowest index;
 * NaN below all else), keep_b in all and in their order; a sequence of at most
 * keep_b keys keeps them.  With per_head every KV head chooses by its own
 * weights (row r of the cache then holds the r-th kept key of each head, of
 * other tokens perhaps: keys carry their positions, so attention over the cache
 * goes on as before); without it all heads keep the same tokens, by the sum of
 * the heads' weights (fp32, in the heads' order).
 *   keep: the most keys that a sequence may keep, >= 1; keep_lens DEVICE int32
 *      [B] or NULL: keep_b, taken into [0, keep] (NULL: keep).  A keep_b below
 *      sinks + recent keeps the sinks first.
 *   kept DEVICE int32 [B, Hkv or 1, keep] out: the logical indexes that stay,
 *      increasing, then -1;  new_lens DEVICE int32 [B] out: min(n, keep_b)
 *      (not kv_lens itself)
 *   out_table NULL: the kept rows of K, V and the weights move to the front of
 *      their own sequence's pages; behind new_lens[b] K and V are what they
 *      were, and the weights up to n become 0, so that keys appended there
 *      begin without any.  Else DEVICE int32 [B, out_width]: they are copied to
 *      the front of the sequence in those pages, which no page_table of the
 *      call may use; nothing else of those pages, and nothing of page_table's,
 *      is written (a page that a sequence is given is to be handed out with
 *      weights of 0).
 * Two sequences must not name the same page when rows move in place, nor two
 * sequences' out_tables.  A length outside [0, width * page_size] or above 2^30
 * is recorded as RA_ERR_DEVICE_BOUNDS and taken as 0 keys; a key on a page
 * outside the cache is recorded, weighs least, and its row is not moved.
 * A copy: the rows' bits do not change.  d of whole 16 bytes, d <= 256; the
 * cache 16-byte aligned with strides of whole 16 bytes (0 is refused, as for
 * the weights).  Capturable; no
 * workspace.  B = 0 does nothing.
 * ------------------------------------------------------------------------ */
ra_status ra_kv_cache_evict(const ra_paged_kv *cache, const ra_paged_weights *weights, const int32_t *page_table,
                            int64_t table_width, const int32_t *kv_lens, int B, int keep, const int32_t *keep_lens,
                            int sinks, int recent, int per_head, const int32_t *out_table, int64_t out_width,
                            int32_t *new_lens, int32_t *kept, void *stream);

/* ------------------------------------------------------------------------
 * ra_delta_rule_fwd / ra_delta_rule_bwd / ra_delta_rule_step  (DEVICE tensors
 * and DEVICE segment arrays)
 *
 * The gated delta rule over packed sequences: the mixer of tokens whose memory
 * is a state of fixed size, S [dk, dv] for each value head.  Token t, with
 * a = exp(g[t]) and b = beta[t]:
 *   S <- a S;   u = b (v - S^T k);   S <- S + k u^T;   out = scale S^T q
 * Value head h reads query and key head h / (Hv / Hk).
 *   q, k DEVICE [T, Hk, dk], v DEVICE [T, Hv, dv] of dtype (rows q_stride,
 *      k_stride, v_stride elements apart); g, beta DEVICE fp32 [T, Hv]
 *      contiguous: the logarithm of the decay (usually <= 0; -inf forgets all,
 *      as does anything below -1e4), and the writing strength
 *   cu_seqlens DEVICE int32 [N+1], non-decreasing, from 0 on; tokens at or
 *      behind cu_seqlens[N] (a padded batch) are left alone: no output and no
 *      gradient is written for them
 *   state DEVICE fp32 [n_slots, Hv, dk, dv] or NULL (zeros): the states ahead
 *      of the sequences; slots DEVICE int32 [N] or NULL (0, 1, ...): sequence
 *      b's place.  A negative slot: the sequence begins at zero and its last
 *      state is dropped.  A slot at or above n_slots is treated so too, and
 *      RA_ERR_DEVICE_BOUNDS is recorded.
 * Forward: out DEVICE [T, Hv, dv] contiguous, of dtype; state_out NULL or
 *   DEVICE fp32 [n_slots, Hv, dk, dv], the states behind the sequences at the
 *   same slots (it may be `state`; two sequences of one call must not name one
 *   slot).
 * Backward: dout DEVICE [T, Hv, dv] of dtype (rows dout_stride apart), dstate
 *   DEVICE fp32 [N, Hv, dk, dv] or NULL (zeros): the gradients of out and of
 *   the last states, by sequence; dq, dk [T, Hk, dk], dv [T, Hv, dv]
 *   contiguous of dtype, dg, dbeta fp32 [T, Hv], dstate0 NULL or fp32
 *   [N, Hv, dk, dv], by sequence.  Nothing of the forward is needed: the
 *   states are computed again.
 * Step: one token of each sequence (T = N, cu_seqlens and state of d unused):
 *   `state` is read and written in place at the slots, which differ from one
 *   another; a sequence without a slot gets output 0.
 * States, sums and gates are fp32, and the products' operands carry 24 bits; out
 * has the same bits with and without state_out.  One rounding of each bf16
 * result; deterministic.  A NaN or an
 * infinity reaches every token of its chunk (64 tokens of a sequence) and all
 * behind it.  Chunks of a sequence with nothing to forget are exact in the
 * same sense at any length.
 * dk and dv 64 or 128; q, k, v, dout and all outputs 16-byte aligned with
 * strides of whole 16 bytes; T <= 2^30, N <= 2^20, N * Hv <= 2^26.
 * workspace DEVICE, 256-byte aligned, >= ra_delta_rule_workspace_bytes(...)
 * (0 for invalid arguments; 48 KB for each chunk of 64 tokens and value head, 272
 * KB for a backward with heads of 128); calls in flight at the same time, and
 * captured graphs that may run so, need workspaces of their own.  Capturable;
 * the arrays' contents may change between replays.  Boundaries that decrease or
 * leave [0, T] are recorded as RA_ERR_DEVICE_BOUNDS and leave all outputs
 * unwritten.
 * ------------------------------------------------------------------------ */
typedef struct ra_delta {
    const void *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;
    const float *g, *beta;
    int64_t T;
    int32_t N, Hk, Hv, dk, dv, dtype;
    const int32_t *cu_seqlens;
    const float *state;
    const int32_t *slots;
    int64_t n_slots;
    float scale;
} ra_delta;
size_t ra_delta_rule_workspace_bytes(int64_t T, int N, int Hk, int Hv, int dk, int dv, int dtype, int bwd);
ra_status ra_delta_rule_fwd(const ra_delta *d, void *out, float *state_out, void *workspace, size_t ws_bytes,
                            void *stream);
ra_status ra_delta_rule_bwd(const ra_delta *d, const void *dout, int64_t dout_stride, const float *dstate, void *dq,
                            void *dk, void *dv, float *dg, float *dbeta, float *dstate0, void *workspace,
                            size_t ws_bytes, void *stream);
ra_status ra_delta_rule_step(const ra_delta *d, float *state, void *out, void *stream);

/* ------------------------------------------------------------------------
 * ra_ring_rank_pairs  (HOST, synchronous)
 *
 * Allowed (query, key) pairs each simulated rank computes over the whole
 * ring: the causal load that zigzag balances ("Question about varlen ring
 * attention", MiniMax-01 #6: causal imbalance; ring-attention-pytorch #20:
 * zigzag spreads it).  window as in ra_varlen_attn_partial (-1 = none).
 * counts HOST [cp] int64.
 * ------------------------------------------------------------------------ */
ra_status ra_ring_rank_pairs(const int32_t *cu_seqlens, int B, int cp, int zz_mode, int causal, int window,
                             int64_t *counts);

/* ------------------------------------------------------------------------
 * ra_ring_plan_stats  (HOST only; no GPU needed)
 *
 * What the tensor-core passes of ra_ring_attn_fwd / bwd visit for a packing
 * (bf16, d = 128; G = Hq / Hkv a power of two dividing 128), found by
 * walking every work item over its range of ring steps with the kernels'
 * own step-to-rank rule and tile classifier (tile-level skipping of fully
 * masked blocks, FlagScale PR #910).  stats HOST int64[RA_PLAN_STATS_N]:
 *   [0] query tiles (128/G tokens x G heads)   [1] key tiles (128 keys)
 *   [2] forward items  [3] dK/dV items  [4] dQ items (all KV heads)
 *   [5] forward visited (query tile, key tile) pairs, one KV head
 *   [6]   of which full (no mask inside)
 *   [7] rows of two-run query tiles  [8] rows of two-run key tiles
 *       (the rows the permutes copy into rank order)
 *   [9] token-pair capacity of the forward's visited pairs
 *       ([5] x 128/G x 128: the tensor work per head group / (2 d G))
 *   exact != 0 (brute force over the visited pairs; else -1):
 *   [10] allowed (query token, key) pairs inside the forward's visited pairs
 *   [11] disallowed pairs among valid rows and keys of "full" pairs
 *   [12] allowed pairs inside the dK/dV pass's visited pairs
 *   [13] allowed pairs inside the dQ pass's visited pairs
 *   [14] dK/dV visited pairs  [15] dQ visited pairs
 *   scheduling model over n_sm SMs, in tile-pair visits per SM (all KV
 *   heads; the ideal is the pass's total visits / n_sm):
 *   [16] forward (persistent CTAs claiming items in order)
 *   [17] dK/dV (one CTA per item, dispatched in order as SMs free up)
 *   [18] dQ (persistent CTAs, static stride over the items)
 *   [19] forward KV steps: KV tiles the forward items of one KV head walk
 *        with a product of either query tile ([5] counts one per query tile)
 * A correct plan covers each allowed pair once in every pass: [10], [12]
 * and [13] equal the sum of ra_ring_rank_pairs, and [11] is 0.
 * ------------------------------------------------------------------------ */
#define RA_PLAN_STATS_N 20
ra_status ra_ring_plan_stats(const int32_t *cu_seqlens, int B, int cp, int zz_mode, int G, int Hkv, int causal,
                             int window, int sched, int exact, int n_sm, int64_t *stats);
/* The same statistics under an interval mask (key_lo / key_hi as in
 * ra_ring_attn_fwd_masked; RA_SCHED_FUSED or RA_SCHED_ALLGATHER). */
ra_status ra_ring_plan_stats_masked(const int32_t *cu_seqlens, int B, int cp, int zz_mode, int G, int Hkv,
                                    const int32_t *key_lo, const int32_t *key_hi, int sched, int exact, int n_sm,
                                    int64_t *stats);

/* Reads and clears the device status word of the current device (waits for
 * `stream` first).  Returns RA_OK, RA_ERR_TIMEOUT or RA_ERR_DEVICE_BOUNDS. */
ra_status ra_get_device_status(void *stream);

/* Self-test of the device-wait guard: launches one CTA that waits on an
 * mbarrier nothing ever arrives at, with a budget of `budget_us`
 * microseconds (1..1000000).  The wait runs out, the kernel records
 * RA_ERR_TIMEOUT in the status word and returns; no copy or MMA is in
 * flight.  Read the result with ra_get_device_status().  Every real kernel
 * uses the same guard (2 s budget) on each of its waits. */
ra_status ra_selftest_wait_timeout(int64_t budget_us, void *stream);

/* ------------------------------------------------------------------------
 * Per-kernel timing (HOST).  While enabled, every kernel launch the library
 * makes is bracketed by two CUDA events recorded on its launching stream.
 * ra_profile_enable(1) clears earlier records; ra_profile_read waits for
 * the recorded events and reports, per kernel name (at most max_kernels,
 * names written as NUL-terminated strings of up to 64 bytes each into
 * `names`), the summed device time in ms and the launch count.  Returns
 * the number of kernels reported, or -1 on error.  Timing adds two event
 * records per launch; keep it off for throughput runs.  Independently of
 * this switch, each timed unit (a kernel launch, or the concurrent backward
 * pair "ra_tc_bwd") is also an NVTX range of the same name pushed on the
 * calling host thread, so a timeline tool shows the phases of a step and,
 * in STEPWISE mode, one range per ring step; with no tool attached the
 * range calls do nothing.
 * ------------------------------------------------------------------------ */
ra_status ra_profile_enable(int on);
int ra_profile_read(int max_kernels, char *names, double *total_ms, int64_t *launches);

const char *ra_status_string(ra_status s);
const char *ra_last_error(void);
const char *ra_version(void);

#ifdef __cplusplus
}
#endif
#endif /* RA_H_ */

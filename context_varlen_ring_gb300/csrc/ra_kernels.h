// ra_kernels.h -- launch interfaces of the library's kernels (host side).
// Included by the C-ABI drivers and by the .cu files that implement them.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "../../include/ra.h"

namespace ra {

// ------------------------------------------------------------ status word
int *device_status_ptr();          // device address of this device's status word
uint64_t wait_budget_ns();         // budget of every device-side wait

// ------------------------------------------------------------ timing
// Brackets one launch with CUDA events on `st` when profiling is enabled.
class ProfScope {
  public:
    ProfScope(const char *name, cudaStream_t st);
    ~ProfScope();

  private:
    int id_ = -1;
    cudaStream_t st_;
};

// ------------------------------------------------------------ permute
struct PermJob {
    const void *src;
    void *dst;
    int64_t row_bytes;
    const uint8_t *only = nullptr;  // T bytes: move just the rows i with only[i] != 0
};
// inverse = 0: dst[i] = src[perm[i]];  inverse = 1: dst[perm[i]] = src[i].
// Up to 4 jobs share one launch (same perm, same T).
cudaError_t launch_permute(const PermJob *jobs, int njobs, const int32_t *perm, int64_t T, int inverse,
                           cudaStream_t st);
// [H, T] fp32: x[h, perm[i]] = y[h, i].
cudaError_t launch_unpermute_cols(const float *y, float *x, const int32_t *perm, int64_t T, int H,
                                  cudaStream_t st);

// ------------------------------------------------------------ merge & misc
constexpr int kMaxMergeParts = 64;
cudaError_t launch_merge(int n, const float *const *outs, const float *const *lses, int64_t Tq, int Hq, int d,
                         void *out, int out_dtype, float *lse_out, cudaStream_t st);
// D[h, t] = sum_c a[t, h, c] * b[t, h, c]   (a, b of dtype; fp32 result)
// Backward preprocess of bf16 tensors with head dim 128, one pass: permute
// the jobs (Q, K, V) and dO (dout -> dout_p, Hq heads) by perm, and
// D[h, p] = sum_c dO[p, h, c] * O[p, h, c] in fp32 at original rows p.
// All pointers and row sizes must be 16-byte aligned (else cudaErrorInvalidValue).
// With dout_only (T bytes) given, dout_p receives just the rows i with
// dout_only[i] != 0 (D is written for every row).
// Copies n bytes from page-locked host memory (mapped into the device's
// address space) to device memory with a kernel, so the copy never queues
// behind other streams' transfers on a copy engine.  src and dst must be
// 16-byte aligned (else cudaErrorInvalidValue).
cudaError_t launch_copy_from_host(const void *src, void *dst, size_t n, cudaStream_t st);
cudaError_t launch_permute_rowdot(const PermJob *jobs, int njobs, const void *dout, void *dout_p, const void *out,
                                  float *D, const int32_t *perm, int64_t T, int Hq, cudaStream_t st,
                                  const uint8_t *dout_only = nullptr);
cudaError_t launch_rowdot(const void *a, const void *b, int dtype, int64_t T, int H, int d, float *D,
                          cudaStream_t st);
// Per (query tile, KV head): 128 columns of -lse*log2(e) (-inf for empty
// rows) then 128 of -D*scale, contiguous (1 KB per tile and head), for the
// key-side backward's bulk copies.
cudaError_t launch_tile_lse_d(const void *qtiles, int n_qtiles, int Hkv, int G, const float *lse, const float *D,
                              int64_t lse_T, float scale, float *out, cudaStream_t st);
// dst (dtype) = src (fp32), n elements.
cudaError_t launch_cast_f32(const float *src, void *dst, int dtype, int64_t n, cudaStream_t st);

// ------------------------------------------------------------ attention
// Where an attention kernel writes its rows.
enum OutMode {
    kOutFinal = 0,    // dtype output at row = position (original order), lse[h*lse_T + position]
    kOutPartial = 1,  // fp32 output at the local row, lse[h*lse_T + local row]
};

// A ring over `cp` simulated ranks.  Query rows of rank r, segment b are
// [qoff[r] + qcul[r*(B+1)+b], qoff[r] + qcul[r*(B+1)+b+1]); key rows of rank s
// likewise with koff/kcul.  Positions (for the causal test and for kOutFinal
// rows) come from qpos / kpos.
struct SimtArgs {
    const void *q, *k, *v;
    int dtype, Hq, Hkv, d;
    int64_t Tq, Tk;
    const int32_t *qoff, *qcul, *qpos;
    const int32_t *koff, *kcul, *kpos;
    int cp, B, t0, t1;
    int causal;
    int window;                        // sliding window (keys at most this far behind), < 0: none
    float scale;
    int out_mode;
    void *out;
    float *lse;
    int64_t lse_T;
};
cudaError_t launch_simt_fwd(const SimtArgs &a, cudaStream_t st);

struct SimtBwdArgs {
    const void *q, *k, *v, *dout;
    int dtype, Hq, Hkv, d;
    int64_t T;                         // rows of the permuted buffers
    const int32_t *off, *cul, *pos;    // ring over cp ranks, q side = k side
    int cp, B, t0, t1;
    int causal;
    int window;                        // sliding window (keys at most this far behind), < 0: none
    float scale;
    const float *lse, *D;              // [Hq, lse_T] indexed by position
    int64_t lse_T;
    float *dq;                         // fp32 [T_orig, Hq, d] at position rows (+=)
    float *dk, *dv;                    // fp32 [T_orig, Hkv, d] at position rows (+=)
};
cudaError_t launch_simt_bwd(const SimtBwdArgs &a, cudaStream_t st);

// Tensor-core forward (bf16, d = 128).
struct TcFwdArgs {
    const void *q, *k, *v;             // permuted buffers
    const void *q_orig, *k_orig, *v_orig;  // nullable: Q / K and V in original order
                                       // (rows = positions); single-run tiles are read from them
    int64_t Tq, Tk;
    int Hq, Hkv, G;
    const void *qtiles, *kvtiles;      // Tile records (two int4 each)
    const int32_t *kv_off;             // [cp*(B+1)+1]
    const void *items;                 // WorkItem records
    int *sched;                        // [2] work counter, zero before the first launch
    int n_items;                       // item count (an upper bound when n_items_dev is given)
    const int *n_items_dev;            // nullable: the item count in device memory
    int cp, B;
    int t0, t1;                        // >= 0: override every item's step range
    int causal;
    int window;                        // sliding window (keys at most this far behind), < 0: none
    const void *qbounds;               // interval masks (else NULL): QBounds per query tile,
    const int32_t *key_lo, *key_hi;    // and each token's key bounds [Tq] at its original position
    float scale;
    int out_mode;
    void *out;
    float *lse;
    int64_t lse_T;
};
cudaError_t launch_tc_fwd(const TcFwdArgs &a, cudaStream_t st);
bool tc_fwd_supported(int dtype, int d, int Hq, int Hkv);

// Tensor-core key-side backward (bf16, d = 128): dK and dV, one CTA per KV
// tile and KV head.  out_mode: 0 bf16 store, 1 fp32 store, 2 fp32 +=.
struct TcBwdArgs {
    const void *q, *k, *v, *dout;      // permuted buffers
    const void *q_orig, *dout_orig;    // nullable pair: Q and dO in original order, read for
                                       // single-run query tiles
    const void *k_orig, *v_orig;       // nullable pair: K and V likewise for KV tiles
    int64_t T;
    int Hq, Hkv, G;
    const void *qtiles, *kvtiles;      // Tile records
    const int32_t *q_off;              // [cp*(B+1)+1]
    const void *items;                 // key-side WorkItem records (qt0 = KV tile)
    int n_items;
    int cp, B;
    int t0, t1;                        // >= 0: override every item's step range
    int causal;
    int window;                        // sliding window (keys at most this far behind), < 0: none
    const void *qbounds;               // interval masks (else NULL), as in TcFwdArgs
    const int32_t *key_lo, *key_hi;
    float scale;
    const float *tile_ld;              // launch_tile_lse_d output for these tiles
    void *dk, *dv;                     // [T, Hkv, d] at original positions
    int out_mode;
};
cudaError_t launch_tc_bwd(const TcBwdArgs &a, cudaStream_t st);

// Tensor-core dQ pass (bf16, d = 128): one CTA per query tile and KV head;
// no atomics.  out_mode: 0 bf16 store, 1 fp32 store, 2 fp32 +=.
struct TcDqArgs {
    const void *q, *k, *v, *dout;      // permuted buffers
    const void *q_orig, *dout_orig;    // nullable pairs, as in TcBwdArgs
    const void *k_orig, *v_orig;
    int64_t T;
    int Hq, Hkv, G;
    const void *qtiles, *kvtiles;
    const int32_t *kv_off;
    const void *items;                 // dQ WorkItem records (qt0 = query tile)
    int n_items;
    int cp, B;
    int t0, t1;
    int causal;
    int window;                        // sliding window (keys at most this far behind), < 0: none
    const void *qbounds;               // interval masks (else NULL), as in TcFwdArgs
    const int32_t *key_lo, *key_hi;
    float scale;
    const float *lse, *D;              // [Hq, lse_T] at original positions
    int64_t lse_T;
    void *dq;                          // [T, Hq, d] at original positions
    int out_mode;
};
cudaError_t launch_tc_dq(const TcDqArgs &a, cudaStream_t st);

// ------------------------------------------------------------ device tile tables
// The tile tables of one partial call built on the device (ra_tile_build.cu):
// query tiles of q_rows rows and KV tiles of 128 rows, at most two position
// runs each, per segment; forward items (pairs of query tiles x KV heads,
// head major), their count in *n_items and the work counter zeroed.  Tables
// sized by the host bound (a tile holds at least one row).  Malformed
// segment boundaries (or, with check_pos, positions outside [0, 2^30)) are
// recorded as RA_ERR_DEVICE_BOUNDS and leave *n_items = 0.
struct DevTileArgs {
    const int32_t *cu_q, *cu_k;        // DEVICE [nseg + 1]
    const int32_t *q_pos, *k_pos;      // DEVICE [Tq], [Tk]; NULL = row index
    int64_t Tq, Tk;
    int nseg, Hkv, q_rows, check_pos;
    void *qtiles, *kvtiles, *items;    // Tile [Tq + nseg], Tile [Tk + nseg], WorkItem [pairs x Hkv]
    int32_t *q_off, *kv_off;           // [nseg + 2]
    int32_t *q_cnt, *k_cnt, *pair_off; // scratch [nseg], [nseg], [nseg + 1]
    int *n_items, *sched;              // 1 int, 2 ints
};
cudaError_t launch_tile_build(const DevTileArgs &a, cudaStream_t st);

// ------------------------------------------------------------ rotary positions, cache append
struct RopeJob {
    const void *x;
    void *y;
    int64_t x_stride, y_stride;        // elements between tokens
    int heads;
    int rotate;                        // 0: copied
    int paged;                         // written to the token's cache row instead of its token row
    int groups;                        // of hpi heads (set by launch_rope)
};
// Travels with the launch (a kernel parameter), so a captured graph keeps it.
struct RopeParams {
    RopeJob jobs[3];
    int njobs, total_heads, d;
    int64_t T;
    const int32_t *pos;                // DEVICE [axes][T]
    int n_pairs, adjacent, inverse;
    int units, rot_units, split;       // set by launch_rope
    int hpi, unit_inv;                 // heads a warp takes at once; 2^16 / units, rounded up
    int stages, stage_bytes, parts, share;  // of the ring kernel: a token's shares, heads a share
    unsigned long long budget_ns;
    // cache rows (cu != NULL): logical index kv_lens[b] - n_b + j through the page table
    const int32_t *cu, *kv_lens, *page_table;
    int64_t table_width, table_keys, n_pages, page_stride, token_stride, head_stride;
    int B, page_size, page_shift;      // page_shift: its log2, or -1
    int *status;
    uint64_t turns[128];               // inv_freq / (2 pi) modulo 1, in units of 2^-64
    uint8_t axis[128];
};
void rope_table(RopeParams &p, const double *inv_freq, const uint8_t *axes, int n_pairs, int adjacent, int inverse);
cudaError_t launch_rope(RopeParams &p, int dtype, cudaStream_t st);

// ------------------------------------------------------------ paged attention
// Families of segments: 0 the sequences' own keys, 1 the groups' prefixes.
// Each (segment, tile of `rt` query rows, KV head) is a unit of ceil(keys / kt)
// key tiles; a unit and its tiles weigh what they cost, and the units form one
// line that the family's `n` CTAs split evenly.  What CTA c computes of a unit
// whose rows start at partial row `base` goes to partial rows base + rt * c on: along the line units and CTAs
// only grow, and no unit has more than rt partial rows, so these never meet.
struct alignas(16) PagedSeg {
    int tok0, n, len, w;               // first query token, query tokens, keys, key tiles
    long long W0, R0;                  // weight of tiles and partial rows ahead of it
};
struct PagedHdr {                      // of each family
    long long W, per;                  // weight in all, weight a CTA
    int err, pad[3];
};
struct PagedFamily {
    int S, rt, kt, n;                  // segments, rows a unit, keys a tile, CTAs
    int rt_log, kt_log;                // (rows and keys are powers of two)
    int halves;                        // units of at most rt / 2 rows: two partials a row, of alternate key tiles
    int least;                         // least weight a CTA (16ths of a tile): less costs more partials than it gains
    PagedHdr *hdr;
    PagedSeg *seg;                     // [S]
    int *start;                        // [n] the segment in which each CTA's run begins
    const int32_t *table;
    int64_t width;
    float *acc, *ml;                   // [partial rows][d], [partial rows][2]: sum p v; running maximum (log2), sum p
};
struct PagedArgs {
    const void *q;
    int64_t q_stride, T;
    int Hq, Hkv, G, d, dtype;
    const void *k, *v;
    int64_t n_pages, page_stride, token_stride, head_stride;
    int page_size, page_shift;         // page_shift: its log2, or -1
    unsigned long long G_inv;          // 2^64 / G, rounded up (G > 1)
    int B, n_groups, causal;
    const int32_t *cu, *kv_lens, *prefix_lens, *groups;
    float scale_log2;
    int here;                          // no plan kernel: every block plans for itself
    PagedFamily f[2];
    void *out;
    int out_dtype;
    float *lse;
    int *status;
};
constexpr int kPagedMostKeys = 1 << 30;  // of a segment: places, tiles and their weights stay within 32 bits
constexpr int kPagedHere = 256;         // most segments of a family that blocks plan for themselves
constexpr int kPagedMaxCtas = 1024;     // of the warp-level and SIMT kernels
constexpr int kPagedMaxWide = 256;      // of the tcgen05 kernel (one an SM)
constexpr int kPagedWideRows = 256;     // its rows a unit
cudaError_t launch_paged_plan(const PagedArgs &a, cudaStream_t st);
// `late`: launched behind the other family's kernel, which it need not wait for
// (it reads the plan only); it then waits before it ends, so that the join,
// which waits for it, finds both families' partials.
cudaError_t launch_paged_simt(const PagedArgs &a, int family, int late, cudaStream_t st);
cudaError_t launch_paged_combine(const PagedArgs &a, cudaStream_t st);
int paged_simt_ctas(int rt, int d);    // CTAs of the SIMT kernel that the current device holds at once
bool paged_mma_supported(int dtype, int d);
int paged_mma_ctas(int rt, int d, int page_size);
cudaError_t launch_paged_mma(const PagedArgs &a, int family, int late, cudaStream_t st);
int paged_sms();                       // SMs of the current device
struct PagedMaps {
    CUtensorMap q, k, v;
    int rows_inner;                    // the cache's rows in a page lie closer than its heads
};
bool paged_tc_maps(const PagedArgs &a, PagedMaps &m);  // false: not a shape of the tcgen05 kernel
cudaError_t launch_paged_tc(const PagedArgs &a, int family, int late, const PagedMaps &m, cudaStream_t st);

// Device-wait self-test (see ra_selftest_wait_timeout).
cudaError_t launch_wait_selftest(uint64_t budget_ns, cudaStream_t st);

}  // namespace ra

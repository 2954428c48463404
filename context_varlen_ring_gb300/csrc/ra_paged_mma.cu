// ra_paged_mma.cu -- paged attention for a few query rows per KV head (bf16,
// d = 64 or 128): warp-level matrix instructions fed by cp.async.
//
// Bound: memory.  A decoding step has G rows (query tokens x the query heads
// of one KV head) against every cached key, 4 d bytes a key and head, each
// used once; tensor work is 2 x 2 d flops per row and key, far below the
// tensor rate even with the rows padded to the 16 of m16n8k16.  So the design
// is about bytes in flight: every warp streams its own 16-key blocks through
// a private two-stage ring (8 KB a stage at d = 128), no warp waits for
// another inside a unit, and rows of any page size are gathered 16 bytes at a
// time.  Scores, maximum, sum and products stay in registers; the warps'
// partials are joined in shared memory when the CTA's run of the unit ends.
//
// With more rows the key tile is shared: up to 32 rows a pair of warps has 16
// rows and half of the keys each, up to 64 every warp has 16 rows and all keys.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "ra_dev.cuh"
#include "ra_kernels.h"
#include "ra_paged.cuh"

namespace ra {
namespace {

using namespace dev;

constexpr int kWarps = 4;
constexpr int kKT = 64;      // keys a tile: 16 for each warp
constexpr int kStages = 2;

__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool there, uint64_t policy) {
    asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst), "l"(src),
                 "r"(there ? 16 : 0), "l"(policy)
                 : "memory");
}
__device__ __forceinline__ void cp16(uint32_t dst, const void *src, uint64_t policy) {
    asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "l"(policy)
                 : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t a, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Shared address of 16-byte chunk c of row r: chunks are exchanged by the
// row's low bits, so that eight rows of one chunk fall into eight bank groups.
// (Row bases are multiples of the row's bytes, so chunk 2 k + b of a row is
// its chunk b's address with bits 5 and up exchanged by k.)
template <int D>
__device__ __forceinline__ uint32_t chunk_at(uint32_t base, int r, int c) {
    return base + (uint32_t)(r * (D * 2) + ((c ^ (r & 7)) << 4));
}

// Where 16 keys from logical index kb on lie: with whole blocks in a page
// (page_size % 16 == 0) the first one's row, the same in every lane; else lane
// i < 16 holds row i's.  -1: none.  Looked up one tile ahead of its use.
template <bool WHOLE>
__device__ __forceinline__ long long find16(const PagedArgs &a, const PagedFamily &f, int s, int len, int kb) {
    if (WHOLE) return paged_row(a, f, s, len, kb);
    const int lane = threadIdx.x & 31;
    return lane < 16 ? paged_row(a, f, s, len, kb + lane) : -1;
}

// Starts the copies of those 16 rows (K and V); rows that are not there are
// filled with zeros, so whatever the cache holds behind a sequence's end never
// meets the products.
template <int D, bool WHOLE>
__device__ __forceinline__ void issue16(const PagedArgs &a, long long off, int live, int h, uint32_t ks, uint32_t vs,
                                        uint64_t policy) {
    constexpr int CPR = D / 8, RPI = 32 / CPR;  // chunks a row, rows a warp instruction
    const int lane = threadIdx.x & 31, c = lane % CPR, r0 = lane / CPR;
    const __nv_bfloat16 *k = static_cast<const __nv_bfloat16 *>(a.k) + h * a.head_stride + c * 8;
    const __nv_bfloat16 *v = static_cast<const __nv_bfloat16 *>(a.v) + h * a.head_stride + c * 8;
    // row i * RPI + r0 lies at (first row's address) ^ (its low bits << 4), + i * RPI rows
    const uint32_t kd = chunk_at<D>(ks, r0, c), vd = chunk_at<D>(vs, r0, c);
    if (WHOLE && off >= 0 && live >= 16) {
        const __nv_bfloat16 *kp = k + off + r0 * a.token_stride, *vp = v + off + r0 * a.token_stride;
#pragma unroll
        for (int i = 0; i < 16 / RPI; ++i) {
            const uint32_t x = (uint32_t)((i * RPI & 7) << 4);
            cp16((kd ^ x) + i * RPI * D * 2, kp, policy);
            cp16((vd ^ x) + i * RPI * D * 2, vp, policy);
            kp += RPI * a.token_stride;
            vp += RPI * a.token_stride;
        }
        return;
    }
    if (WHOLE && off < 0) live = 0;
#pragma unroll
    for (int i = 0; i < 16 / RPI; ++i) {
        const int r = i * RPI + r0;
        const uint32_t x = (uint32_t)((i * RPI & 7) << 4);
        const long long o = WHOLE ? off + r * a.token_stride : __shfl_sync(0xffffffffu, off, r);
        const bool there = WHOLE ? r < live : o >= 0;
        cp16((kd ^ x) + i * RPI * D * 2, k + (there ? o : 0), there, policy);
        cp16((vd ^ x) + i * RPI * D * 2, v + (there ? o : 0), there, policy);
    }
}

template <int D>
struct Rows {
    uint32_t q[D / 16][4];  // A fragments of the 16 query rows
    float o[D / 8][4];      // sum p v of rows lane / 4 and lane / 4 + 8
    float m[2], l[2];       // running maximum (log2), sum p of the lane's own keys
    int lim[2];             // keys the rows see
};

// One block of 16 keys for 16 rows: S = Q K^T, the running maximum, P in
// bf16, O += P V.  The sums use the unrounded values.  With WHOLE_P P is two
// bf16 parts, a product each (2^-15 of P is lost, not 2^-8): single tokens are
// bound by memory and the results lose nothing beside their own rounding (64
// ragged requests: error against 64 bits 0.0021 -> 0.0017, 77.8 -> 78.3 us;
// one request of 8192 keys 14.0 -> 14.6 us).  With shared key tiles (17 rows
// and more) P is rounded, as in the tcgen05 kernel and the packed ring: there
// the products show (drafts' own keys, 43.9 -> 46.4 us).
constexpr float kLeast = 9.5367431640625e-7f;  // 2^-20
template <int D, bool WHOLE_P>
__device__ __forceinline__ void block16(Rows<D> &w, uint32_t ks, uint32_t vs, int kb, bool masked, float scale_log2) {
    const int lane = threadIdx.x & 31, id = lane >> 3, l8 = lane & 7;
    float s[2][4] = {};
    const uint32_t ka = chunk_at<D>(ks, (id >> 1) * 8 + l8, id & 1);
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
        uint32_t b[4];
        ldsm4(ka ^ (k << 5), b);
        mma16816(s[0], w.q[k], b[0], b[1]);
        mma16816(s[1], w.q[k], b[2], b[3]);
    }
#pragma unroll
    for (int n = 0; n < 2; ++n) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            s[n][e] *= scale_log2;
            if (masked && kb + n * 8 + (lane & 3) * 2 + (e & 1) >= w.lim[e >> 1]) s[n][e] = -INFINITY;
        }
    }
    float mn[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        float x = fmaxf(fmaxf(s[0][2 * r], s[0][2 * r + 1]), fmaxf(s[1][2 * r], s[1][2 * r + 1]));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
        mn[r] = fmaxf(w.m[r], x);
    }
    if (__any_sync(0xffffffffu, mn[0] > w.m[0] || mn[1] > w.m[1])) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const float alpha = mn[r] == -INFINITY ? 1.f : ex2_approx(w.m[r] - mn[r]);
            w.m[r] = mn[r];
            w.l[r] *= alpha;
#pragma unroll
            for (int n = 0; n < D / 8; ++n) {
                w.o[n][2 * r] *= alpha;
                w.o[n][2 * r + 1] *= alpha;
            }
        }
    }
    uint32_t p[4], rest[4] = {};
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const float use = w.m[r] == -INFINITY ? 0.f : w.m[r];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const float p0 = ex2_approx(s[n][2 * r] - use), p1 = ex2_approx(s[n][2 * r + 1] - use);
            w.l[r] += p0 + p1;
            if (!WHOLE_P) {
                p[2 * n + r] = pack_bf16x2(p0, p1);
            } else {
                // the upper halves, and what they cut off: 2^-20 of the weight at least, so that an infinite value stays
                // one, and nothing of a weight of zero, so that the largest value behind a mask adds nothing
                const uint32_t u0 = __float_as_uint(p0), u1 = __float_as_uint(p1);
                p[2 * n + r] = __byte_perm(u0, u1, 0x7632);
                rest[2 * n + r] = pack_bf16x2(fmaxf(p0 - __uint_as_float(u0 & 0xffff0000u), p0 * kLeast),
                                              fmaxf(p1 - __uint_as_float(u1 & 0xffff0000u), p1 * kLeast));
            }
        }
    }
    const uint32_t va = chunk_at<D>(vs, (id & 1) * 8 + l8, id >> 1);
#pragma unroll
    for (int n = 0; n < D / 16; ++n) {
        uint32_t b[4];
        ldsm4t(va ^ (n << 5), b);
        mma16816(w.o[2 * n], p, b[0], b[1]);
        mma16816(w.o[2 * n + 1], p, b[2], b[3]);
        if (WHOLE_P) {
            mma16816(w.o[2 * n], rest, b[0], b[1]);
            mma16816(w.o[2 * n + 1], rest, b[2], b[3]);
        }
    }
}

// Rows a unit: 16, 32 or 64, in tiles of 16; KW = 64 / ROWS warps have a tile
// of rows in common and the blocks of keys in turn.
template <int D, int ROWS>
constexpr size_t mma_smem() {
    return (size_t)kWarps * kStages * 2 * 16 * D * 2 + (ROWS == 64 ? 0 : kWarps * 16 * sizeof(float2));
}

template <int D, int ROWS, bool WHOLE>
__global__ void __launch_bounds__(kWarps * 32, 3)
    paged_mma_kernel(const __grid_constant__ PagedArgs a, int fi, int late) {
    constexpr int KW = 64 / ROWS;
    constexpr uint32_t kBlk = 16 * D * 2;          // bytes of 16 rows
    constexpr uint32_t kStage = kWarps * 2 * kBlk;  // K blocks of the warps, then V blocks
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t base = smem_u32(smem);
    const PagedFamily &f = a.f[fi];
    if (!late) pdl_wait();
    pdl_launch();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    __shared__ PlanShared plan;
    // Each warp's place in the CTA's run, and its unit in hand and the next
    // one: in shared memory, where they hold no registers in the loop over keys.
    __shared__ PagedWalk place[kWarps];
    __shared__ PagedUnit units[kWarps][2];
    {
        const PagedWalk k = paged_begin<kWarps * 32>(a, f, fi, plan);
        if (lane == 0) place[warp] = k;
        __syncwarp();
    }
    const uint64_t policy = l2_evict_first();
    int it = 0;                      // key tiles so far: tile i lies in stage i % kStages
    // this warp's 16 keys of tile t
    auto find = [&](const PagedUnit &u, int t) { return find16<WHOLE>(a, f, u.s, u.len, t * kKT + warp * 16); };
    auto issue = [&](const PagedUnit &u, long long off, int t, int i) {
        const uint32_t st = base + (uint32_t)i % kStages * kStage + warp * kBlk;
        issue16<D, WHOLE>(a, off, u.len - (t * kKT + warp * 16), u.h, st, st + kWarps * kBlk, policy);
    };
    auto sync_tile = [&]() {  // a warp alone with its keys waits for nobody
        if (KW == kWarps)
            __syncwarp();
        else
            __syncthreads();
    };
    long long ahead = -1;  // the next tile's place, when it is of the unit in hand
    for (int i = 0;; ++i) {
        bool more;
        {
            PagedWalk k = place[warp];
            PagedUnit next;
            more = paged_unit(a, f, fi, k, next);
            __syncwarp();
            if (lane == 0) {
                place[warp] = k;
                if (more) units[warp][i & 1] = next;
            }
            __syncwarp();
        }
        const PagedUnit &nu = units[warp][i & 1];
        if (i == 0) {
            if (!more) break;
            issue(nu, find(nu, nu.t0), nu.t0, 0);
            cp_commit();
            if (nu.t0 + 1 < nu.t1) ahead = find(nu, nu.t0 + 1);
            continue;
        }
        const PagedUnit &u = units[warp][(i & 1) ^ 1];
        Rows<D> w;
        int lo, hi;  // the warp's rows: the fewest and the most keys any of them sees
        {
            const int R = u.n * a.G, r0 = u.r0 + warp / KW * 16;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int row = r0 + (lane >> 2) + 8 * r;
                // (padding rows pass for rows that see all keys: no masks for them, their results are dropped)
                w.lim[r] = row < R ? paged_limit(a, u, fi, row) : u.len;
                w.m[r] = -INFINITY;
                w.l[r] = 0.f;
                const bool ok = row < R;
                const int tok = paged_token(a, row);
                const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(a.q) +
                                         (ok ? (int64_t)(u.tok0 + tok) * a.q_stride +
                                                   (int64_t)(u.h * a.G + row - tok * a.G) * D : 0) + (lane & 3) * 2;
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    w.q[k][r] = ok ? *reinterpret_cast<const uint32_t *>(q + k * 16) : 0u;
                    w.q[k][2 + r] = ok ? *reinterpret_cast<const uint32_t *>(q + k * 16 + 8) : 0u;
                }
            }
            if (r0 >= R) w.lim[0] = w.lim[1] = 0;  // a warp without rows only loads
        }
        lo = min(w.lim[0], w.lim[1]);
        hi = max(w.lim[0], w.lim[1]);
#pragma unroll
        for (int o = 16; o >= 4; o >>= 1) {
            lo = min(lo, __shfl_xor_sync(0xffffffffu, lo, o));
            hi = max(hi, __shfl_xor_sync(0xffffffffu, hi, o));
        }
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) w.o[n][e] = 0.f;
        const int64_t slot = u.base + (int64_t)blockIdx.x * ROWS;
        const int rows = u.rows;
        for (int t = u.t0, t1 = u.t1; t < t1; ++t, ++it) {
            // the next tile is on its way while this one is used, the next unit's first one too
            if (t + 1 < t1) {
                issue(u, ahead, t + 1, it + 1);
                if (t + 2 < t1) ahead = find(u, t + 2);
            } else if (more) {
                issue(nu, find(nu, nu.t0), nu.t0, it + 1);
                if (nu.t0 + 1 < nu.t1) ahead = find(nu, nu.t0 + 1);
            }
            cp_commit();
            cp_wait<1>();
            sync_tile();
            const uint32_t st = base + (uint32_t)it % kStages * kStage;
#pragma unroll 1
            for (int b = warp % KW * (kWarps / KW), e = b + kWarps / KW; b < e; ++b) {
                const int kb = t * kKT + b * 16;
                if (kb < hi)
                    block16<D, ROWS == 16>(w, st + b * kBlk, st + (kWarps + b) * kBlk, kb, kb + 16 > lo, a.scale_log2);
            }
            sync_tile();  // the stage may be filled again
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {  // the four lanes of a row hold different keys
            w.l[r] += __shfl_xor_sync(0xffffffffu, w.l[r], 1);
            w.l[r] += __shfl_xor_sync(0xffffffffu, w.l[r], 2);
        }
        if (KW == 1) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int row = warp * 16 + (lane >> 2) + 8 * r;
                if (row >= rows) continue;
                const int64_t at = slot + row;
#pragma unroll
                for (int n = 0; n < D / 8; ++n)
                    *reinterpret_cast<float2 *>(f.acc + at * D + n * 8 + (lane & 3) * 2) =
                        make_float2(w.o[n][2 * r], w.o[n][2 * r + 1]);
                if ((lane & 3) == 0) *reinterpret_cast<float2 *>(f.ml + at * 2) = make_float2(w.m[r], w.l[r]);
            }
        } else {
            // the warps' partials, joined in the stage that was used last (the other one is being filled);
            // float c of a row lies at c ^ 8 (row & 7), to spread the rows over the banks
            float *all = reinterpret_cast<float *>(smem + (uint32_t)(it - 1) % kStages * kStage);
            float2 *ml = reinterpret_cast<float2 *>(smem + kStages * kStage);  // [kWarps][16]
            __syncthreads();  // every warp is done with the stage
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int row = (lane >> 2) + 8 * r;
#pragma unroll
                for (int n = 0; n < D / 8; ++n)
                    *reinterpret_cast<float2 *>(all + (warp * 16 + row) * D +
                                                ((n * 8 + (lane & 3) * 2) ^ (8 * (row & 7)))) =
                        make_float2(w.o[n][2 * r], w.o[n][2 * r + 1]);
                if ((lane & 3) == 0) ml[warp * 16 + row] = make_float2(w.m[r], w.l[r]);
            }
            __syncthreads();
#pragma unroll 1
            for (int row = warp; row < rows; row += kWarps) {
                const int j0 = row / 16 * KW * 16 + row % 16;  // its row in the first of its tile's warps
                float M = -INFINITY, L = 0.f, acc[D / 32];
#pragma unroll
                for (int j = 0; j < KW; ++j) M = fmaxf(M, ml[j0 + j * 16].x);
#pragma unroll
                for (int e = 0; e < D / 32; ++e) acc[e] = 0.f;
#pragma unroll
                for (int j = 0; j < KW; ++j) {
                    const float2 v = ml[j0 + j * 16];
                    const float wt = M == -INFINITY ? 0.f : ex2_approx(v.x - M);
                    L += wt * v.y;
#pragma unroll
                    for (int e = 0; e < D / 32; ++e)
                        acc[e] = fmaf(wt, all[(j0 + j * 16) * D + ((lane + 32 * e) ^ (8 * (row & 7)))], acc[e]);
                }
                const int64_t at = slot + row;
#pragma unroll
                for (int e = 0; e < D / 32; ++e) f.acc[at * D + lane + 32 * e] = acc[e];
                if (lane == 0) *reinterpret_cast<float2 *>(f.ml + at * 2) = make_float2(M, L);
            }
            __syncthreads();  // the stage may be filled again
        }
        if (!more) break;
    }
    if (late) pdl_wait();  // the join waits for this kernel only: it must not end ahead of its predecessor
}

template <int D, int ROWS, bool WHOLE>
cudaError_t mma_launch(const PagedArgs *a, int fi, int late, int *ctas, cudaStream_t st) {
    static_assert(kStages == 2 && (size_t)kWarps * 16 * D * 4 <= (size_t)kWarps * 2 * 16 * D * 2,
                  "one tile ahead; the joined rows lie over one stage");
    auto kernel = paged_mma_kernel<D, ROWS, WHOLE>;
    constexpr size_t smem = mma_smem<D, ROWS>();
    static LaunchFit fit;
    const cudaError_t e = fit.prepare((const void *)kernel, kWarps * 32, smem, ctas);
    if (e != cudaSuccess || ctas) return e;
    return launch_pdl(kernel, a->f[fi].n, kWarps * 32, smem, st, *a, fi, late);
}

template <int D, int ROWS>
cudaError_t mma_by_page(int page, const PagedArgs *a, int fi, int late, int *ctas, cudaStream_t st) {
    return page % 16 == 0 ? mma_launch<D, ROWS, true>(a, fi, late, ctas, st)
                          : mma_launch<D, ROWS, false>(a, fi, late, ctas, st);
}

template <int D>
cudaError_t mma_by_rows(int rt, int page, const PagedArgs *a, int fi, int late, int *ctas, cudaStream_t st) {
    return rt == 16   ? mma_by_page<D, 16>(page, a, fi, late, ctas, st)
           : rt == 32 ? mma_by_page<D, 32>(page, a, fi, late, ctas, st)
                      : mma_by_page<D, 64>(page, a, fi, late, ctas, st);
}

cudaError_t mma_by_shape(int rt, int d, int page, const PagedArgs *a, int fi, int late, int *ctas, cudaStream_t st) {
    if (d == 128) return mma_by_rows<128>(rt, page, a, fi, late, ctas, st);
    if (d == 64) return mma_by_rows<64>(rt, page, a, fi, late, ctas, st);
    return cudaErrorInvalidValue;
}

}  // namespace

bool paged_mma_supported(int dtype, int d) { return dtype == RA_BF16 && (d == 64 || d == 128); }

int paged_mma_ctas(int rt, int d, int page_size) {
    int n = 0;
    if (mma_by_shape(rt, d, page_size, nullptr, 0, 0, &n, nullptr) != cudaSuccess || n < 1) n = 1;
    return std::min(kPagedMaxCtas, n * paged_sms());
}

cudaError_t launch_paged_mma(const PagedArgs &a, int fi, int late, cudaStream_t st) {
    return mma_by_shape(a.f[fi].rt, a.d, a.page_size, &a, fi, late, nullptr, st);
}

}  // namespace ra

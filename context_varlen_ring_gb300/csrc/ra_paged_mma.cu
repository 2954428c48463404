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
// With 17 to 32 rows a warp keeps two row tiles for each of its keys (Q then
// comes from shared memory); with more, where the tcgen05 kernel does not take
// the shape, the warps go over the rows and share the key tile (64 rows a CTA).
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

template <int D, int MT>
struct Rows {
    uint32_t q[MT == 1 ? D / 16 : 1][4];  // A fragments of the 16 query rows (two row tiles read theirs from shared memory)
    float o[MT][D / 8][4];                // sum p v of rows 16 i + lane / 4 and + 8
    float m[MT][2], l[MT][2];             // running maximum (log2), sum p of the lane's own keys
    int lim[MT][2];                       // keys the rows see
};

// One block of 16 keys for MT tiles of 16 rows: S = Q K^T, the running
// maximum, P in bf16 (rounded once: the products' inputs; the sums use the
// unrounded values), O += P V.  Each key and value fragment serves every tile.
template <int D, int MT>
__device__ __forceinline__ void block16(Rows<D, MT> &w, uint32_t qs, uint32_t ks, uint32_t vs, int kb, bool masked,
                                        float scale_log2) {
    const int lane = threadIdx.x & 31, id = lane >> 3, l8 = lane & 7;
    float s[MT][2][4] = {};
    const uint32_t ka = chunk_at<D>(ks, (id >> 1) * 8 + l8, id & 1);
    const uint32_t qa = chunk_at<D>(qs, (id & 1) * 8 + l8, id >> 1);
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
        uint32_t b[4];
        ldsm4(ka ^ (k << 5), b);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            if (MT == 1) {
                mma16816(s[i][0], w.q[k % (MT == 1 ? D / 16 : 1)], b[0], b[1]);
                mma16816(s[i][1], w.q[k % (MT == 1 ? D / 16 : 1)], b[2], b[3]);
            } else {
                uint32_t q[4];
                ldsm4((qa ^ (k << 5)) + i * 16 * D * 2, q);
                mma16816(s[i][0], q, b[0], b[1]);
                mma16816(s[i][1], q, b[2], b[3]);
            }
        }
    }
    uint32_t p[MT][4];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
#pragma unroll
        for (int n = 0; n < 2; ++n) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                s[i][n][e] *= scale_log2;
                if (masked && kb + n * 8 + (lane & 3) * 2 + (e & 1) >= w.lim[i][e >> 1]) s[i][n][e] = -INFINITY;
            }
        }
        float mn[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            float x = fmaxf(fmaxf(s[i][0][2 * r], s[i][0][2 * r + 1]), fmaxf(s[i][1][2 * r], s[i][1][2 * r + 1]));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
            mn[r] = fmaxf(w.m[i][r], x);
        }
        if (__any_sync(0xffffffffu, mn[0] > w.m[i][0] || mn[1] > w.m[i][1])) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const float alpha = mn[r] == -INFINITY ? 1.f : ex2_approx(w.m[i][r] - mn[r]);
                w.m[i][r] = mn[r];
                w.l[i][r] *= alpha;
#pragma unroll
                for (int n = 0; n < D / 8; ++n) {
                    w.o[i][n][2 * r] *= alpha;
                    w.o[i][n][2 * r + 1] *= alpha;
                }
            }
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const float use = w.m[i][r] == -INFINITY ? 0.f : w.m[i][r];
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const float p0 = ex2_approx(s[i][n][2 * r] - use), p1 = ex2_approx(s[i][n][2 * r + 1] - use);
                w.l[i][r] += p0 + p1;
                p[i][2 * n + r] = pack_bf16x2(p0, p1);
            }
        }
    }
    const uint32_t va = chunk_at<D>(vs, (id & 1) * 8 + l8, id >> 1);
#pragma unroll
    for (int n = 0; n < D / 16; ++n) {
        uint32_t b[4];
        ldsm4t(va ^ (n << 5), b);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            mma16816(w.o[i][2 * n], p[i], b[0], b[1]);
            mma16816(w.o[i][2 * n + 1], p[i], b[2], b[3]);
        }
    }
}

// Rows a unit: 16 or 32 with the warps over the keys (ROWS), 64 with the warps over the rows.
template <int D, int ROWS>
constexpr size_t mma_smem() {
    return (size_t)kWarps * kStages * 2 * 16 * D * 2 +
           (ROWS == 64 ? 0 : kWarps * ROWS * sizeof(float2) + (ROWS == 32 ? 32 * D * 2 : 0));
}

template <int D, int ROWS, bool WHOLE>
__global__ void __launch_bounds__(kWarps * 32, ROWS == 32 ? 2 : 3)
    paged_mma_kernel(const __grid_constant__ PagedArgs a, int fi, int late) {
    constexpr bool WIDE = ROWS == 64;
    constexpr int MT = ROWS == 32 ? 2 : 1;
    constexpr uint32_t kBlk = 16 * D * 2;          // bytes of 16 rows
    constexpr uint32_t kStage = kWarps * 2 * kBlk;  // K blocks of the warps, then V blocks
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t base = smem_u32(smem);
    const PagedFamily &f = a.f[fi];
    if (!late) pdl_wait();
    pdl_launch();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    __shared__ PlanShared plan;
    PagedWalk walk = paged_begin<kWarps * 32>(a, f, fi, plan);
    if (walk.x >= walk.x1) {
        if (late) pdl_wait();
        return;
    }
    const uint64_t policy = l2_evict_first();
    int it = 0;                      // key tiles so far: tile i lies in stage i % kStages
    // this warp's 16 keys of tile t of the walk's segment
    auto find = [&](int t) { return find16<WHOLE>(a, f, walk.s, walk.g.len, t * kKT + warp * 16); };
    auto issue = [&](long long off, int h, int t, int i) {
        const uint32_t st = base + (uint32_t)i % kStages * kStage + warp * kBlk;
        issue16<D, WHOLE>(a, off, walk.g.len - (t * kKT + warp * 16), h, st, st + kWarps * kBlk, policy);
    };
    PagedUnit u = paged_unit(a, f, fi, walk);
    issue(find(u.t0), u.h, u.t0, 0);
    cp_commit();
    long long ahead = u.t0 + 1 < u.t1 ? find(u.t0 + 1) : -1;  // the next tile's place, when it is of this unit
    const uint32_t qs = base + kStages * kStage;               // two row tiles: Q [32][D], then the joins' statistics
    for (bool more = true; more;) {
        Rows<D, MT> w;
        int lo, hi;  // the warp's rows: the fewest and the most keys any of them sees
        {
            const PagedSeg &g = walk.g;
            const int R = g.n * a.G, r0 = u.r0 + (WIDE ? warp * 16 : 0);
            auto q_at = [&](int row) {
                return static_cast<const __nv_bfloat16 *>(a.q) + (int64_t)(g.tok0 + row / a.G) * a.q_stride +
                       (int64_t)(u.h * a.G + row % a.G) * D;
            };
#pragma unroll
            for (int i = 0; i < MT; ++i) {
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int row = r0 + 16 * i + (lane >> 2) + 8 * r;
                    // (padding rows pass for rows that see all keys: no masks for them, their results are dropped)
                    w.lim[i][r] = row < R ? paged_limit(a, g, fi, row) : g.len;
                    w.m[i][r] = -INFINITY;
                    w.l[i][r] = 0.f;
                    if (MT == 1) {
                        const bool ok = row < R;
                        const __nv_bfloat16 *q = (ok ? q_at(row) : static_cast<const __nv_bfloat16 *>(a.q)) + (lane & 3) * 2;
#pragma unroll
                        for (int k = 0; k < D / 16; ++k) {
                            w.q[k % (MT == 1 ? D / 16 : 1)][r] = ok ? *reinterpret_cast<const uint32_t *>(q + k * 16) : 0u;
                            w.q[k % (MT == 1 ? D / 16 : 1)][2 + r] =
                                ok ? *reinterpret_cast<const uint32_t *>(q + k * 16 + 8) : 0u;
                        }
                    }
                }
            }
            if (MT > 1) {
                for (int c = threadIdx.x; c < 16 * MT * (D / 8); c += kWarps * 32) {
                    const int row = c / (D / 8), ch = c % (D / 8);
                    uint4 v = make_uint4(0, 0, 0, 0);
                    if (r0 + row < R) v = *reinterpret_cast<const uint4 *>(q_at(r0 + row) + ch * 8);
                    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(chunk_at<D>(qs, row, ch)), "r"(v.x),
                                 "r"(v.y), "r"(v.z), "r"(v.w)
                                 : "memory");
                }
                __syncthreads();
            }
            if (WIDE && r0 >= R) w.lim[0][0] = w.lim[0][1] = 0;  // a warp without rows only loads
        }
        lo = min(w.lim[0][0], w.lim[0][1]);
        hi = max(w.lim[0][0], w.lim[0][1]);
        if (MT > 1) {
            lo = min(lo, min(w.lim[MT - 1][0], w.lim[MT - 1][1]));
            hi = max(hi, max(w.lim[MT - 1][0], w.lim[MT - 1][1]));
        }
#pragma unroll
        for (int o = 16; o >= 4; o >>= 1) {
            lo = min(lo, __shfl_xor_sync(0xffffffffu, lo, o));
            hi = max(hi, __shfl_xor_sync(0xffffffffu, hi, o));
        }
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int n = 0; n < D / 8; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) w.o[i][n][e] = 0.f;
        const int64_t slot = u.base + (int64_t)blockIdx.x * ROWS;
        const int rows = u.rows;
        for (int t = u.t0, t1 = u.t1; t < t1; ++t, ++it) {
            // the next tile is on its way while this one is used, the next unit's first one too
            if (t + 1 < t1) {
                issue(ahead, u.h, t + 1, it + 1);
                if (t + 2 < t1) ahead = find(t + 2);
            } else {
                walk.x += t1 - u.t0;
                more = walk.x < walk.x1;
                if (more) {
                    u = paged_unit(a, f, fi, walk);
                    issue(find(u.t0), u.h, u.t0, it + 1);
                    if (u.t0 + 1 < u.t1) ahead = find(u.t0 + 1);
                }
            }
            cp_commit();
            cp_wait<1>();
            if (WIDE)
                __syncthreads();
            else
                __syncwarp();
            const uint32_t st = base + (uint32_t)it % kStages * kStage;
#pragma unroll 1
            for (int b = WIDE ? 0 : warp; b < (WIDE ? kWarps : warp + 1); ++b) {
                const int kb = t * kKT + b * 16;
                if (kb < hi)
                    block16<D, MT>(w, qs, st + b * kBlk, st + (kWarps + b) * kBlk, kb, kb + 16 > lo, a.scale_log2);
            }
            // the stage may be filled again
            if (WIDE)
                __syncthreads();
            else
                __syncwarp();
        }
#pragma unroll
        for (int i = 0; i < MT; ++i) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {  // the four lanes of a row hold different keys
                w.l[i][r] += __shfl_xor_sync(0xffffffffu, w.l[i][r], 1);
                w.l[i][r] += __shfl_xor_sync(0xffffffffu, w.l[i][r], 2);
            }
        }
        if (WIDE) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int row = warp * 16 + (lane >> 2) + 8 * r;
                if (row >= rows) continue;
                const int64_t at = slot + row;
#pragma unroll
                for (int n = 0; n < D / 8; ++n)
                    *reinterpret_cast<float2 *>(f.acc + at * D + n * 8 + (lane & 3) * 2) =
                        make_float2(w.o[0][n][2 * r], w.o[0][n][2 * r + 1]);
                if ((lane & 3) == 0) *reinterpret_cast<float2 *>(f.ml + at * 2) = make_float2(w.m[0][r], w.l[0][r]);
            }
        } else {
            // the warps' partials, 16 rows at a time, joined in the stage that was used last (the other one is
            // being filled); float c of a row lies at c ^ 8 (row & 7), to spread the rows over the banks
            float *all = reinterpret_cast<float *>(smem + (uint32_t)(it - 1) % kStages * kStage);
            float2 *ml = reinterpret_cast<float2 *>(smem + kStages * kStage + (MT > 1 ? 32 * D * 2 : 0));  // [kWarps][16]
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                __syncthreads();  // every warp is done with the stage
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int row = (lane >> 2) + 8 * r;
#pragma unroll
                    for (int n = 0; n < D / 8; ++n)
                        *reinterpret_cast<float2 *>(all + (warp * 16 + row) * D +
                                                    ((n * 8 + (lane & 3) * 2) ^ (8 * (row & 7)))) =
                            make_float2(w.o[i][n][2 * r], w.o[i][n][2 * r + 1]);
                    if ((lane & 3) == 0) ml[warp * 16 + row] = make_float2(w.m[i][r], w.l[i][r]);
                }
                __syncthreads();
                for (int row = warp; row < 16 && 16 * i + row < rows; row += kWarps) {
                    float M = -INFINITY, L = 0.f, acc[D / 32];
#pragma unroll
                    for (int j = 0; j < kWarps; ++j) M = fmaxf(M, ml[j * 16 + row].x);
#pragma unroll
                    for (int e = 0; e < D / 32; ++e) acc[e] = 0.f;
#pragma unroll
                    for (int j = 0; j < kWarps; ++j) {
                        const float2 v = ml[j * 16 + row];
                        const float wt = M == -INFINITY ? 0.f : ex2_approx(v.x - M);
                        L += wt * v.y;
#pragma unroll
                        for (int e = 0; e < D / 32; ++e)
                            acc[e] = fmaf(wt, all[(j * 16 + row) * D + ((lane + 32 * e) ^ (8 * (row & 7)))], acc[e]);
                    }
                    const int64_t at = slot + 16 * i + row;
#pragma unroll
                    for (int e = 0; e < D / 32; ++e) f.acc[at * D + lane + 32 * e] = acc[e];
                    if (lane == 0) *reinterpret_cast<float2 *>(f.ml + at * 2) = make_float2(M, L);
                }
            }
            __syncthreads();  // the stage may be filled again
        }
    }
    if (late) pdl_wait();  // the join waits for this kernel only: it must not end ahead of its predecessor
}

template <int D, int ROWS, bool WHOLE>
cudaError_t mma_launch(const PagedArgs *a, int fi, int late, int *ctas, cudaStream_t st) {
    static_assert(kStages == 2 && (size_t)kWarps * 16 * D * 4 <= (size_t)kWarps * 2 * 16 * D * 2,
                  "one tile ahead; the joined rows lie over one stage");
    auto kernel = paged_mma_kernel<D, ROWS, WHOLE>;
    constexpr size_t smem = mma_smem<D, ROWS>();
    cudaError_t e = cudaFuncSetAttribute((const void *)kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    if (ctas) return cudaOccupancyMaxActiveBlocksPerMultiprocessor(ctas, kernel, kWarps * 32, smem);
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

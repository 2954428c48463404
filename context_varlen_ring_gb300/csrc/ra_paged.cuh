// ra_paged.cuh -- what the paged-attention kernels share on the device: the
// walk of a CTA along its run of key tiles, the keys a row sees, and the page table.
#pragma once

#include <utility>

#include "ra_kernels.h"
#include "ra_serve.cuh"

namespace ra {
namespace dev {

// x / y of non-negative numbers, in 32 bits wherever they fit (a 64-bit
// division is some hundred instructions).
__device__ __forceinline__ long long paged_div(long long x, long long y) {
    return ((x | y) >> 32) == 0 ? (long long)((uint32_t)x / (uint32_t)y) : x / y;
}

// Query token of a row, row / G: exact for rows of 32 bits, by one product.
__device__ __forceinline__ int paged_token(const PagedArgs &a, int row) {
    return a.G == 1 ? row : (int)__umul64hi((unsigned)row, a.G_inv);
}
// Page of a key, and its row in it.
__device__ __forceinline__ int paged_page(const PagedArgs &a, int key) {
    return a.page_shift >= 0 ? key >> a.page_shift : key / a.page_size;
}

// Partial rows of a tile of `rows` query rows.
__device__ __forceinline__ int paged_alloc(const PagedFamily &f, int rows) {
    return f.halves && 2 * rows <= f.rt ? 2 * rows : rows;
}

struct PagedUnit {
    int s, tok0, n, len; // its segment
    int r0, rows, h;     // first query row in the segment, query rows, KV head
    int t0, t1;          // the CTA's key tiles in it
    long long base;      // first partial row (of CTA 0)
};

// Segment s of a family from the call's arrays (W0 and R0 left to the plan);
// false, and an empty one, where they are not as they must be.
__device__ __forceinline__ bool paged_record(const PagedArgs &a, const PagedFamily &f, int fi, int s, PagedSeg &g) {
    const int len = fi ? a.prefix_lens[s] : a.kv_lens[s];
    const int b0 = fi ? a.groups[s] : s, b1 = fi ? a.groups[s + 1] : s + 1;
    // (loaded whatever the others say, so that no load waits for another's check)
    int c0 = a.cu[min(max(b0, 0), a.B)], c1 = a.cu[min(max(b1, 0), a.B)];
    const bool fine = b0 >= 0 && b1 >= b0 && b1 <= a.B && len >= 0 && len <= f.width * a.page_size &&
                      len <= kPagedMostKeys && c0 >= 0 && c1 >= c0 && c1 <= a.T;
    if (!fine) c0 = c1 = 0;
    g.tok0 = c0;
    g.n = c1 - c0;
    g.len = fine ? len : 0;
    g.w = g.n > 0 ? (g.len + f.kt - 1) >> f.kt_log : 0;
    g.W0 = g.R0 = 0;
    return fine;
}
// What a unit and its key tiles weigh, in sixteenths of a warp-level tile: a
// unit takes its own cost (queries, join, partial) and then its tiles, so a run
// that goes on into another unit has fewer tiles for it.  Of the tcgen05 kernel,
// a tile for two row tiles takes 1.75 us, one of alternating tiles for a single
// row tile 1.0 to 1.4 (bound by its softmax, or by memory), a unit about 4.
struct PagedCost {
    int tile, unit;
};
__device__ __forceinline__ PagedCost paged_cost(const PagedArgs &a, const PagedFamily &f, const PagedSeg &g) {
    return PagedCost{!f.halves ? 16 : g.n * a.G * 2 > f.rt ? 48 : 32, f.halves ? 96 : 32};
}
__device__ __forceinline__ int paged_all(const PagedSeg &g, const PagedCost &c) {  // (at most 2^24 tiles)
    return g.w ? g.w * c.tile + c.unit : 0;
}
// The first tile of a unit that begins at or behind place `at` of it: a tile
// belongs to the run in which it begins.
__device__ __forceinline__ int paged_tile(int at, const PagedCost &c) {
    const unsigned x = (unsigned)max(at - c.unit + c.tile - 1, 0) >> 4;
    return (int)(c.tile == 48 ? x / 3 : c.tile == 32 ? x >> 1 : x);
}
// The weight of all its units, and its partial rows.  (n * G < 2^31.)
__device__ __forceinline__ long long paged_tiles(const PagedArgs &a, const PagedFamily &f, const PagedSeg &g) {
    return (long long)((g.n * a.G + f.rt - 1) >> f.rt_log) * a.Hkv * paged_all(g, paged_cost(a, f, g));
}
// The weight of a CTA's run.
__device__ __forceinline__ long long paged_per(const PagedFamily &f, long long W) {
    return max((long long)f.least, paged_div(W + f.n - 1, f.n));
}
__device__ __forceinline__ long long paged_rows(const PagedArgs &a, const PagedFamily &f, const PagedSeg &g) {
    const int R = g.n * a.G, full = R & -f.rt;
    return (long long)a.Hkv * (full + paged_alloc(f, R - full));
}

// A CTA's run of the line, and its place in it: the segment and the unit.
struct PagedWalk {
    long long x, x1;
    int s;
    PagedSeg g;
};

// The plan kernel's record of a segment.  Its results are read past L1, which
// may hold an earlier call's.
__device__ __forceinline__ PagedSeg paged_seg(const PagedFamily &f, int s) {
    const int4 *p = reinterpret_cast<const int4 *>(f.seg + s);
    const int4 a = __ldcg(p), b = __ldcg(p + 1);
    PagedSeg g;
    g.tok0 = a.x;
    g.n = a.y;
    g.len = a.z;
    g.w = a.w;
    g.W0 = ((long long)b.y << 32) | (unsigned)b.x;
    g.R0 = ((long long)b.w << 32) | (unsigned)b.z;
    return g;
}

// Up to kPagedHere segments are planned by every block for itself, from the
// call's arrays: a scan over THREADS threads, which costs less than a launch
// ahead of all others and the loads that depend on it (one request of 8192
// keys: 19.6 us with the plan kernel, 15.7 without).  Finds the segment with
// tiles at place blockIdx.x * per (want < 0), or segment `want`; per = 0 where
// an array is not as it must be.
struct PlanShared {
    long long w[32], r[32];
    PagedSeg g;
    int s, bad[32];
};
// Barrier of the block's first THREADS threads (of all of them: 0).
template <int THREADS, int BAR>
__device__ __forceinline__ void plan_sync() {
    if (BAR == 0)
        __syncthreads();
    else
        asm volatile("bar.sync %0, %1;" ::"n"(BAR), "n"(THREADS) : "memory");
}
template <int THREADS, int BAR = 0>
__device__ __forceinline__ long long paged_plan_here(const PagedArgs &a, const PagedFamily &f, int fi, int want,
                                                     PlanShared &sh, long long &W) {
    constexpr int K = (kPagedHere + THREADS - 1) / THREADS;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    PagedSeg g[K];
    long long gw[K], gr[K], w = 0, r = 0;  // of each segment, and of the thread's
    int bad = 0;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int s = threadIdx.x * K + k;
        gw[k] = gr[k] = 0;
        if (s < f.S) {
            bad |= !paged_record(a, f, fi, s, g[k]);
            gw[k] = paged_tiles(a, f, g[k]);
            gr[k] = paged_rows(a, f, g[k]);
        }
        w += gw[k];
        r += gr[k];
    }
    long long wi = w, ri = r;  // inclusive over the warp
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, wi, o), y = __shfl_up_sync(0xffffffffu, ri, o);
        if (lane >= o) {
            wi += x;
            ri += y;
        }
    }
    bad = __any_sync(0xffffffffu, bad);
    if (lane == 31) {
        sh.w[warp] = wi;
        sh.r[warp] = ri;
        sh.bad[warp] = bad;
    }
    plan_sync<THREADS, BAR>();
    long long w0 = wi - w, r0 = ri - r;
    W = 0;
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i) {
        if (i < warp) {
            w0 += sh.w[i];
            r0 += sh.r[i];
        }
        W += sh.w[i];
        bad |= sh.bad[i];
    }
    const long long per = paged_per(f, W);
    if (bad) {
        if (threadIdx.x == 0) record_status(a.status, RA_ERR_DEVICE_BOUNDS);
        W = 0;
    }
    const long long x = blockIdx.x * per;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int s = threadIdx.x * K + k;
        if (s >= f.S) break;
        if (want < 0 ? x >= w0 && x < w0 + gw[k] : s == want) {
            g[k].W0 = w0;
            g[k].R0 = r0;
            sh.g = g[k];
            sh.s = s;
        }
        w0 += gw[k];
        r0 += gr[k];
    }
    plan_sync<THREADS, BAR>();
    return bad ? 0 : per;
}

// The run of this CTA (x >= x1: none), by the plan kernel's results or its own.
__device__ __forceinline__ PagedWalk paged_planned(const PagedFamily &f) {
    PagedWalk k;
    const long long per = __ldcg(&f.hdr->per), W = __ldcg(&f.hdr->W);
    k.s = __ldcg(f.start + blockIdx.x);  // (not meant for a CTA without a run)
    k.x = blockIdx.x * per;
    k.x1 = min(W, k.x + per);
    if (k.x < k.x1) k.g = paged_seg(f, k.s);
    return k;
}
template <int THREADS, int BAR = 0>
__device__ __forceinline__ PagedWalk paged_begin(const PagedArgs &a, const PagedFamily &f, int fi, PlanShared &sh) {
    PagedWalk k;
    if (a.here) {
        long long W;
        const long long per = paged_plan_here<THREADS, BAR>(a, f, fi, -1, sh, W);
        k.x = blockIdx.x * per;
        k.x1 = min(W, k.x + per);
        k.s = sh.s;  // (not meant for a CTA without a run)
        k.g = sh.g;
        return k;
    }
    return paged_planned(f);
}

// The CTA's next unit and its tiles there; false where its run has no more.
// Row tiles are outermost in a segment, so CTAs an equal share of the line
// apart read the same keys for different rows at about the same time (from L2).
__device__ __forceinline__ bool paged_unit(const PagedArgs &a, const PagedFamily &f, int fi, PagedWalk &k, PagedUnit &u) {
    while (k.x < k.x1) {
        for (long long end; (end = k.g.W0 + paged_tiles(a, f, k.g)) <= k.x;) {
            ++k.s;
            if (a.here) {
                const long long rows = k.g.R0 + paged_rows(a, f, k.g);
                paged_record(a, f, fi, k.s, k.g);
                k.g.W0 = end;
                k.g.R0 = rows;
            } else {
                k.g = paged_seg(f, k.s);
            }
        }
        const long long rel = k.x - k.g.W0;
        const PagedCost cost = paged_cost(a, f, k.g);
        const int all = paged_all(k.g, cost);
        const int lu = (int)paged_div(rel, all), rtile = lu < a.Hkv ? 0 : lu / a.Hkv;
        const int from = (int)(rel - (long long)lu * all), to = (int)min((long long)all, from + (k.x1 - k.x));
        k.x += to - from;
        u.t0 = paged_tile(from, cost);
        u.t1 = paged_tile(to, cost);
        if (u.t0 >= u.t1) continue;  // the run ends inside a tile that another one began
        u.s = k.s;
        u.tok0 = k.g.tok0;
        u.n = k.g.n;
        u.len = k.g.len;
        u.h = lu - rtile * a.Hkv;
        u.r0 = rtile << f.rt_log;
        u.rows = min(f.rt, k.g.n * a.G - u.r0);
        u.base = k.g.R0 + (long long)u.r0 * a.Hkv + (long long)u.h * paged_alloc(f, u.rows);
        return true;
    }
    return false;
}

// Keys that row `row` of the segment sees: all of a prefix, the causal part
// of the own keys (a row behind the segment's last sees none).
template <typename Seg>
__device__ __forceinline__ int paged_limit(const PagedArgs &a, const Seg &g, int family, int row) {
    if (row >= g.n * a.G) return 0;
    return family || !a.causal ? g.len : g.len - g.n + paged_token(a, row) + 1;
}

// Element offset of key `i`'s row (head 0), or -1 where there is none: behind
// the length, or on a page outside the cache (recorded).
__device__ __forceinline__ int64_t paged_row(const PagedArgs &a, const PagedFamily &f, int s, int len, int i) {
    if (i >= len) return -1;
    const int pi = paged_page(a, i);
    const int pg = __ldg(f.table + (int64_t)s * f.width + pi);
    if (pg < 0 || pg >= a.n_pages) {
        record_status(a.status, RA_ERR_DEVICE_BOUNDS);
        return -1;
    }
    return pg * a.page_stride + (int64_t)(i - pi * a.page_size) * a.token_stride;
}

// Programmatic launches: a kernel's prologue runs beside its predecessor's
// end.  pdl_wait returns when the predecessor's results can be read;
// pdl_launch lets the successor's CTAs start where there is room.
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

}  // namespace dev

// Launches `kernel` on `st` as a programmatic successor of the kernel ahead of it.
template <typename... P, typename... A>
cudaError_t launch_pdl(void (*kernel)(P...), unsigned grid, unsigned block, size_t smem, cudaStream_t st, A &&...args) {
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t c{};
    c.gridDim = dim3(grid);
    c.blockDim = dim3(block);
    c.dynamicSmemBytes = smem;
    c.stream = st;
    c.attrs = &at;
    c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, kernel, std::forward<A>(args)...);
}

}  // namespace ra

// ra_paged.cuh -- what the paged-attention kernels share on the device: the
// walk of a CTA along its run of key tiles, the keys a row sees, and the page table.
#pragma once

#include <utility>

#include "ra_kernels.h"
#include "ra_paged_split.h"
#include "ra_serve.cuh"

namespace ra {
namespace dev {

// Query token of a row, row / G: exact for rows of 32 bits, by one product.
__device__ __forceinline__ int paged_token(const PagedArgs &a, int row) {
    return a.G == 1 ? row : (int)__umul64hi((unsigned)row, a.G_inv);
}
// Page of a key, and its row in it.
__device__ __forceinline__ int paged_page(const PagedArgs &a, int key) {
    return a.page_shift >= 0 ? key >> a.page_shift : key / a.page_size;
}

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
__device__ __forceinline__ bool paged_unit(const PagedArgs &a, const PagedFamily &f, int fi, PagedWalk &k, PagedUnit &u) {
    return paged_walk(a, f, k, u, [&](PagedWalk &w, long long end) {
        ++w.s;
        if (a.here) {
            const long long rows = w.g.R0 + paged_rows(a, f, w.g);
            paged_record(a, f, fi, w.s, w.g);
            w.g.W0 = end;
            w.g.R0 = rows;
        } else {
            w.g = paged_seg(f, w.s);
        }
    });
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

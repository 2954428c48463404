// ra_paged.cuh -- what the paged-attention kernels share on the device: the
// place of a CTA's run of key tiles, the keys a row sees, and the page table.
#pragma once

#include <utility>

#include "ra_dev.cuh"
#include "ra_kernels.h"

namespace ra {
namespace dev {

// The segment whose tiles hold place x of the line (x < cumW[S]).
__device__ __forceinline__ int paged_find(const PagedFamily &f, long long x) {
    int lo = 0, hi = f.S - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (f.cumW[mid + 1] <= x)
            lo = mid + 1;
        else
            hi = mid;
    }
    return lo;
}

// Partial rows of a tile of `rows` query rows.
__device__ __forceinline__ int paged_alloc(const PagedFamily &f, int rows) {
    return f.halves && 2 * rows <= f.rt ? 2 * rows : rows;
}

struct PagedUnit {
    int r0, rows, h;     // first query row in the segment, query rows, KV head
    int t0, t1;          // the CTA's key tiles in it
    long long base;      // first partial row (of CTA 0)
};

// The unit at place x of segment s, and the CTA's part of it up to place x1.
// Row tiles are outermost, so CTAs an equal share of the line apart read the
// same keys for different rows at about the same time (from L2).
__device__ __forceinline__ PagedUnit paged_unit(const PagedArgs &a, const PagedFamily &f, const PagedSeg &g, int s,
                                                long long x, long long x1) {
    const long long rel = x - f.cumW[s];
    const int lu = (int)(rel / g.w), rtile = lu / a.Hkv;
    PagedUnit u;
    u.t0 = (int)(rel - (long long)lu * g.w);
    u.t1 = (int)min((long long)g.w, u.t0 + (x1 - x));
    u.h = lu - rtile * a.Hkv;
    u.r0 = rtile * f.rt;
    u.rows = min(f.rt, g.n * a.G - u.r0);
    u.base = f.cumR[s] + (long long)u.r0 * a.Hkv + (long long)u.h * paged_alloc(f, u.rows);
    return u;
}

// Keys that row `row` of the segment sees: all of a prefix, the causal part
// of the own keys (a row behind the segment's last sees none).
__device__ __forceinline__ int paged_limit(const PagedArgs &a, const PagedSeg &g, int family, int row) {
    if (row >= g.n * a.G) return 0;
    return family || !a.causal ? g.len : g.len - g.n + row / a.G + 1;
}

// Element offset of key `i`'s row (head 0), or -1 where there is none: behind
// the length, or on a page outside the cache (recorded).
__device__ __forceinline__ int64_t paged_row(const PagedArgs &a, const PagedFamily &f, int s, int len, int i) {
    if (i >= len) return -1;
    const int pg = __ldg(f.table + (int64_t)s * f.width + i / a.page_size);
    if (pg < 0 || pg >= a.n_pages) {
        record_status(a.status, RA_ERR_DEVICE_BOUNDS);
        return -1;
    }
    return pg * a.page_stride + (int64_t)(i % a.page_size) * a.token_stride;
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

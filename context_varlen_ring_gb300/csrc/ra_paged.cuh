// ra_paged.cuh -- what the paged-attention kernels share on the device: the
// walk of a CTA along its run of key tiles, the keys a row sees, and the page table.
#pragma once

#include <utility>

#include "ra_dev.cuh"
#include "ra_kernels.h"

namespace ra {
namespace dev {

// x / y of non-negative numbers, in 32 bits wherever they fit (a 64-bit
// division is some hundred instructions).
__device__ __forceinline__ long long paged_div(long long x, long long y) {
    return ((x | y) >> 32) == 0 ? (long long)((uint32_t)x / (uint32_t)y) : x / y;
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

// A CTA's run of the line, and its place in it: the segment and the unit.
struct PagedWalk {
    long long x, x1;
    int s;
    PagedSeg g;
};

// The run of this CTA (x == x1: none).  The plan's results are read past L1,
// which may hold an earlier call's.
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
__device__ __forceinline__ PagedWalk paged_begin(const PagedFamily &f) {
    const long long per = __ldcg(&f.hdr->per), W = __ldcg(&f.hdr->W);
    PagedWalk k;
    k.s = __ldcg(f.start + blockIdx.x);  // (not meant for a CTA without a run)
    k.x = blockIdx.x * per;
    k.x1 = min(W, k.x + per);
    if (k.x < k.x1) k.g = paged_seg(f, k.s);
    return k;
}

// The unit at the walk's place (in the next segment with tiles, where the last
// one's are done), and the CTA's part of it.  Row tiles are outermost in a
// segment, so CTAs an equal share of the line apart read the same keys for
// different rows at about the same time (from L2).
__device__ __forceinline__ PagedUnit paged_unit(const PagedArgs &a, const PagedFamily &f, PagedWalk &k) {
    auto tiles = [&]() { return (long long)((k.g.n * a.G + f.rt - 1) / f.rt) * a.Hkv * k.g.w; };
    while (k.g.W0 + tiles() <= k.x) k.g = paged_seg(f, ++k.s);
    const long long rel = k.x - k.g.W0;
    const int lu = (int)paged_div(rel, k.g.w), rtile = lu / a.Hkv;
    PagedUnit u;
    u.t0 = (int)(rel - (long long)lu * k.g.w);
    u.t1 = (int)min((long long)k.g.w, u.t0 + (k.x1 - k.x));
    u.h = lu - rtile * a.Hkv;
    u.r0 = rtile * f.rt;
    u.rows = min(f.rt, k.g.n * a.G - u.r0);
    u.base = k.g.R0 + (long long)u.r0 * a.Hkv + (long long)u.h * paged_alloc(f, u.rows);
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
    const int pi = a.page_shift >= 0 ? i >> a.page_shift : i / a.page_size;
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

// ra_paged.cuh -- what the paged-attention kernels share on the device: the
// place of a CTA's run of key tiles, the keys a row sees, and the page table.
#pragma once

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

struct PagedUnit {
    int unit, rtile, h;  // the unit's number, its tile of query rows, its KV head
    int t0, t1;          // the CTA's key tiles in it
};

// The unit at place x of segment s, and the CTA's part of it up to place x1.
// Row tiles are outermost, so CTAs an equal share of the line apart read the
// same keys for different rows at about the same time (from L2).
__device__ __forceinline__ PagedUnit paged_unit(const PagedArgs &a, const PagedFamily &f, const PagedSeg &g, int s,
                                                long long x, long long x1) {
    const long long rel = x - f.cumW[s];
    const int lu = (int)(rel / g.w);
    PagedUnit u;
    u.t0 = (int)(rel - (long long)lu * g.w);
    u.t1 = (int)min((long long)g.w, u.t0 + (x1 - x));
    u.unit = f.cumU[s] + lu;
    u.rtile = lu / a.Hkv;
    u.h = lu - u.rtile * a.Hkv;
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

}  // namespace dev
}  // namespace ra

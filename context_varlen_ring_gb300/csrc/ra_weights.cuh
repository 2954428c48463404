// ra_weights.cuh -- what the key-weight kernels share: the line of all
// segments' tiles, a key's place in the cache, and a query row's place among them.
#pragma once

#include <cuda_runtime.h>

#include "ra_dev.cuh"
#include "ra_keep.h"
#include "ra_kernels.h"

namespace ra {
namespace weights {

using namespace dev;

constexpr int kSegs = 1024;  // segments that a CTA lines up at a time

__device__ __forceinline__ int token_of(const WeightArgs &a, int row) {
    return a.G == 1 ? row : (int)__umul64hi((unsigned)row, a.G_inv);
}

// A segment: own keys of a sequence, or the keys of a prefix (behind the B sequences).
struct Segment {
    int tok0, n, len;
};
__device__ __forceinline__ bool segment(const WeightArgs &a, int s, Segment &g) {
    const int f = s >= a.B, i = s - (f ? a.B : 0);
    const int len = f ? a.prefix_lens[i] : a.kv_lens[i];
    const int b0 = f ? a.groups[i] : i, b1 = f ? a.groups[i + 1] : i + 1;
    const int c0 = a.cu[min(max(b0, 0), a.B)], c1 = a.cu[min(max(b1, 0), a.B)];
    const bool fine = b0 >= 0 && b1 >= b0 && b1 <= a.B && len >= 0 && len <= a.width[f] * a.page_size &&
                      len <= kPagedMostKeys && c0 >= 0 && c1 >= c0 && c1 <= a.T;
    g.tok0 = c0;
    g.n = fine ? c1 - c0 : 0;
    g.len = fine ? len : 0;
    return fine;
}

struct Line {
    int at[kSegs + 1];  // tiles ahead of each segment
    long long warp[32];
};
// Lines up the segments from s0 on; their tiles of 2^k keys, or -1 where any segment is not as it must be (or the
// tiles are more than any memory holds).
// By the block's first THREADS threads, of ALL (which all call it).
template <int THREADS, int ALL = THREADS>
__device__ __forceinline__ int line_up(const WeightArgs &a, int s0, int k, Line &sh) {
    constexpr int PER = kSegs / THREADS;
    const int tid = threadIdx.x, lane = tid & 31, S = a.B + a.n_groups;
    int n[PER], bad = 0;
    long long sum = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int s = s0 + tid * PER + i;
        Segment g;
        n[i] = 0;
        if (s < S && tid < THREADS) {
            bad |= !segment(a, s, g);
            n[i] = g.n > 0 ? (g.len + (1 << k) - 1) >> k : 0;
        }
        sum += n[i];
    }
    long long inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += x;
    }
    __syncthreads();
    if (lane == 31 && tid < THREADS) sh.warp[tid >> 5] = inc;
    bad = __syncthreads_or(bad);
    long long at = inc - sum, all = 0;
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i) {
        if (i < (tid >> 5)) at += sh.warp[i];
        all += sh.warp[i];
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        if (ALL > THREADS && tid >= THREADS) break;
        sh.at[tid * PER + i] = (int)at;
        at += n[i];
    }
    if (tid == THREADS - 1) sh.at[kSegs] = (int)all;
    __syncthreads();
    return bad || all > INT32_MAX ? -1 : (int)all;
}
// The segment of a tile on the line.
__device__ __forceinline__ int find(const Line &sh, int tile) {
    int lo = 0, hi = kSegs;
    while (hi - lo > 1) {
        const int m = (lo + hi) >> 1;
        if (sh.at[m] <= tile)
            lo = m;
        else
            hi = m;
    }
    return lo;
}

// Page and row of a key of segment s; false: on no page of the cache (recorded).
__device__ __forceinline__ bool place(const WeightArgs &a, int s, int key, int64_t &page, int &row) {
    const int f = s >= a.B, i = s - (f ? a.B : 0);
    const int pi = a.page_shift >= 0 ? key >> a.page_shift : key / a.page_size;
    const int p = __ldg(a.table[f] + (int64_t)i * a.width[f] + pi);
    page = p;
    row = key - pi * a.page_size;
    if (p >= 0 && p < a.n_pages) return true;
    record_status(a.status, RA_ERR_DEVICE_BOUNDS);
    return false;
}

// A row's offset in the exponent, -lse in base 2; -inf (nothing is added) behind the segment's rows and where the row
// saw no key.
__device__ __forceinline__ float row_lse(const WeightArgs &a, const Segment &g, int h, int row) {
    if (row >= g.n * a.G) return -INFINITY;
    const int t = token_of(a, row);
    const float x = __ldg(a.lse + (int64_t)(h * a.G + row - t * a.G) * a.T + g.tok0 + t);
    return x == -INFINITY ? -INFINITY : -x * 1.4426950408889634f;
}

// Keys of the segment that a row sees.
__device__ __forceinline__ int limit_of(const WeightArgs &a, const Segment &g, bool own, int row) {
    return own && a.causal ? g.len - g.n + token_of(a, row) + 1 : g.len;
}

}  // namespace weights
}  // namespace ra

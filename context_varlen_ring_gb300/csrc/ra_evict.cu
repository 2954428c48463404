// ra_evict.cu -- eviction from the paged cache: of a sequence's n keys the
// first `sinks`, the last `recent` and the heaviest of the rest stay, `keep`
// in all, in their order; their rows move to the front.
//
// Two kernels.  The choice is a search for the weight of the last key that
// stays, digit by digit over weights mapped to integers of the same order (11,
// 11 and 10 bits: a block's histogram of a digit in shared memory, the digit
// found in it by a sum from the top), and then one pass over the keys that
// writes the places of those above it, and of the first ones equal to it.  A
// long cache of few sequences is split over a cluster of CTAs, whose
// histograms are added through distributed shared memory.  The move is a copy,
// bound by memory.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "ra_dev.cuh"
#include "ra_keep.h"
#include "ra_kernels.h"
#include "ra_serve.cuh"

namespace ra {
namespace {

namespace cg = cooperative_groups;
using namespace dev;

constexpr int kThreads = 1024;
constexpr int kBins = 2048;
constexpr int kHeld = 24576;  // keys of a CTA held in shared memory; more are read again in each pass

// Weights as unsigned integers of the same order: NaN lowest, -0 as 0.
__device__ __forceinline__ uint32_t ordered(float x) {
    if (x != x) return 0;
    const uint32_t b = __float_as_uint(x == 0.f ? 0.f : x);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// Page and row of a key; false: on no page of the cache (recorded).
__device__ __forceinline__ bool place(const EvictArgs &a, const int32_t *table, int64_t width, int b, int key, int64_t &page,
                                      int &row) {
    const int pi = a.page_shift >= 0 ? key >> a.page_shift : key / a.page_size;
    row = key - pi * a.page_size;
    const int p = pi < width ? __ldg(table + b * width + pi) : -1;
    page = p;
    if (p >= 0 && p < a.n_pages) return true;
    record_status(a.status, RA_ERR_DEVICE_BOUNDS);
    return false;
}

__device__ __forceinline__ uint32_t weight_key(const EvictArgs &a, int b, int h, int i) {
    int64_t page;
    int row;
    if (!place(a, a.table, a.width, b, i, page, row)) return 0;
    const float *w = a.w + page * a.w_page + row * a.w_token;
    if (a.H > 1 || a.Hkv == 1) return ordered(w[h * a.w_head]);
    float s = w[0];
    for (int j = 1; j < a.Hkv; ++j) s += w[j * a.w_head];
    return ordered(s);
}

struct ChooseSmem {
    int bins[kBins];
    int warp[32];
    int above, digit;         // of the search
    int gt, eq;               // this CTA's keys above the threshold, and equal to it
    uint32_t held[1];         // (as many as the launch has room for)
};

__global__ void __launch_bounds__(kThreads) evict_choose_kernel(const EvictArgs a, int room) {
    extern __shared__ __align__(16) uint8_t raw[];
    ChooseSmem &sm = *reinterpret_cast<ChooseSmem *>(raw);
    cg::cluster_group cluster = cg::this_cluster();
    const int ranks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int pair = blockIdx.x / ranks, b = pair / a.H, h = pair % a.H;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int n = a.kv_lens[b], keep = a.keep;
    if (a.keep_lens) keep = min(max(a.keep_lens[b], 0), a.keep);
    int32_t *kept = a.kept + (int64_t)pair * a.keep;
    if (n < 0 || n > a.most) {
        if (tid == 0) record_status(a.status, RA_ERR_DEVICE_BOUNDS);
        n = 0;
    }
    const int left = min(n, keep);
    if (h == 0 && rank == 0 && tid == 0) a.new_lens[b] = left;
    const int step = ranks * kThreads, me = rank * kThreads + tid;
    for (int i = left + me; i < a.keep; i += step) kept[i] = -1;
    if (n <= keep) {
        for (int i = me; i < n; i += step) kept[i] = i;
        return;  // (the whole cluster)
    }
    // what stays whatever its weight: the sinks first, then as many of the last as there is room for
    const int first = min(a.sinks, left), last = min(a.recent, left - first);
    for (int i = me; i < first; i += step) kept[i] = i;
    for (int i = me; i < last; i += step) kept[left - last + i] = n - last + i;
    const int want = left - first - last;  // of the keys [first, n - last)
    if (want == 0) return;
    const int mid = n - last - first, per = (mid + ranks - 1) / ranks;
    const int at0 = first + min(mid, rank * per), cnt = first + min(mid, (rank + 1) * per) - at0;
    const bool held = per <= room;
    auto key_at = [&](int i) { return held ? sm.held[i] : weight_key(a, b, h, at0 + i); };
    if (held)
        for (int i = tid; i < cnt; i += kThreads) sm.held[i] = weight_key(a, b, h, at0 + i);
    // the threshold: its digits from the top, and how many of the keys above it are still wanted
    uint32_t prefix = 0, mask = 0;
    int need = want;
    for (int d = 0; d < 3; ++d) {
        const int shift = d == 0 ? 21 : d == 1 ? 10 : 0, bits = d == 2 ? 10 : 11;
        for (int i = tid; i < kBins; i += kThreads) sm.bins[i] = 0;
        __syncthreads();
        for (int i0 = 0; i0 < cnt; i0 += kThreads) {
            const int i = i0 + tid;
            const uint32_t x = i < cnt ? key_at(i) : 0;
            const bool in = i < cnt && (x & mask) == prefix;
            const int digit = in ? (int)(x >> shift) & ((1 << bits) - 1) : -1;
            // lanes of one digit (weights of 0, mostly) are added at once
            int same;
            __match_all_sync(0xffffffffu, digit, &same);
            if (same) {
                if (lane == 0 && digit >= 0) atomicAdd(&sm.bins[digit], 32);
            } else if (digit >= 0) {
                atomicAdd(&sm.bins[digit], 1);
            }
        }
        cluster.sync();
        // two bins a thread, the highest first: counts of the cluster, and their sum from the top
        int c[2] = {0, 0};
        const int top = kBins - 2 - 2 * tid;
        for (int r = 0; r < ranks; ++r) {
            const int2 x = *reinterpret_cast<const int2 *>(cluster.map_shared_rank(&sm.bins[0], r) + top);
            c[0] += x.y;
            c[1] += x.x;
        }
        int sum = c[0] + c[1];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += x;
        }
        if (lane == 31) sm.warp[warp] = sum;
        __syncthreads();
        int above = sum - c[0] - c[1];
        for (int w = 0; w < warp; ++w) above += sm.warp[w];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            if (above < need && above + c[e] >= need) {
                sm.above = above;
                sm.digit = top + 1 - e;
            }
            above += c[e];
        }
        cluster.sync();  // (and no CTA clears its bins before all have read them)
        need -= sm.above;
        prefix |= (uint32_t)sm.digit << shift;
        mask |= (uint32_t)((1 << bits) - 1) << shift;
        __syncthreads();
    }
    // this CTA's keys above the threshold and equal to it, and those of the CTAs ahead of it
    int gt = 0, eq = 0;
    for (int i = tid; i < cnt; i += kThreads) {
        const uint32_t x = key_at(i);
        gt += x > prefix;
        eq += x == prefix;
    }
    if (tid == 0) sm.gt = sm.eq = 0;
    __syncthreads();
    gt = __reduce_add_sync(0xffffffffu, gt);
    eq = __reduce_add_sync(0xffffffffu, eq);
    if (lane == 0) {
        atomicAdd(&sm.gt, gt);
        atomicAdd(&sm.eq, eq);
    }
    cluster.sync();
    int gt0 = 0, eq0 = 0;
    for (int r = 0; r < rank; ++r) {
        gt0 += *cluster.map_shared_rank(&sm.gt, r);
        eq0 += *cluster.map_shared_rank(&sm.eq, r);
    }
    // of the equal ones, the first `need` stay: a key's place is the count of those above ahead of it, and of the equal
    // ones ahead of it as far as they stay
    for (int i0 = 0; i0 < cnt; i0 += kThreads) {
        const int i = i0 + tid;
        const uint32_t x = i < cnt ? key_at(i) : 0;
        const bool g = i < cnt && x > prefix, e = i < cnt && x == prefix;
        const uint32_t bg = __ballot_sync(0xffffffffu, g), be = __ballot_sync(0xffffffffu, e), below = (1u << lane) - 1;
        if (lane == 0) sm.warp[warp] = __popc(bg) << 16 | __popc(be);
        __syncthreads();
        int ahead = 0, all = 0;
#pragma unroll 8
        for (int w = 0; w < 32; ++w) {
            const int y = sm.warp[w];
            if (w < warp) ahead += y;
            all += y;
        }
        const int ga = gt0 + (ahead >> 16) + __popc(bg & below), ea = eq0 + (ahead & 0xffff) + __popc(be & below);
        if (g || (e && ea < need)) kept[first + ga + min(ea, need)] = at0 + i;
        gt0 += all >> 16;
        eq0 += all & 0xffff;
        __syncthreads();
    }
    cluster.sync();  // (no CTA ends while another reads its counts)
}

// ------------------------------------------------------------ the move
constexpr int kMoveThreads = 256;

// To other pages: every row and head by itself, 16 bytes a thread.
__global__ void __launch_bounds__(kMoveThreads) evict_copy_kernel(const EvictArgs a) {
    const int vecs = a.row_bytes / 16, share = 2 * vecs;  // of one row and head: K, then V
    const int per = kMoveThreads / share > 0 ? kMoveThreads / share : 1;
    const int b = blockIdx.y, left = a.new_lens[b];
    const int64_t total = (int64_t)left * a.Hkv;
    const int lane = threadIdx.x % share;
    if ((int)threadIdx.x >= per * share) return;
    for (int64_t u = (int64_t)blockIdx.x * per + threadIdx.x / share; u < total; u += (int64_t)gridDim.x * per) {
        const int j = (int)(u / a.Hkv), h = (int)(u - (int64_t)j * a.Hkv);
        const int i = __ldg(a.kept + ((int64_t)b * a.H + (a.H > 1 ? h : 0)) * a.keep + j);
        int64_t ps, pd;
        int rs, rd;
        if (!place(a, a.table, a.width, b, i, ps, rs) || !place(a, a.out_table, a.out_width, b, j, pd, rd)) continue;
        const int64_t src = (ps * a.page_stride + rs * a.token_stride + h * a.head_stride) * a.esize;
        const int64_t dst = (pd * a.page_stride + rd * a.token_stride + h * a.head_stride) * a.esize;
        char *base = static_cast<char *>(lane < vecs ? a.k : a.v) + (lane % vecs) * 16;
        *reinterpret_cast<uint4 *>(base + dst) = *reinterpret_cast<const uint4 *>(base + src);
        if (lane == 0)
            a.w[pd * a.w_page + rd * a.w_token + h * a.w_head] = a.w[ps * a.w_page + rs * a.w_token + h * a.w_head];
    }
}

// In place: kept key j comes from a place at or behind j, and places only grow, so a batch of rows may be written once
// all of it is read: every row that it overwrites was read in this batch or before.  A CTA walks one head's batches for
// some columns of K or of V.
constexpr int kBatch = 8;  // 16-byte pieces a thread
__global__ void __launch_bounds__(kMoveThreads) evict_shift_kernel(const EvictArgs a, int cols) {
    const int vecs = a.row_bytes / 16 / cols;  // pieces of a row that this CTA moves
    const int col = blockIdx.x % cols, which = blockIdx.x / cols % 2, pair = blockIdx.x / (2 * cols);
    const int b = pair / a.Hkv, h = pair % a.Hkv, left = a.new_lens[b];
    const int per = kMoveThreads / vecs, tid = threadIdx.x, r0 = tid / vecs, c = (col * vecs + tid % vecs) * 16;
    const int32_t *kept = a.kept + ((int64_t)b * a.H + (a.H > 1 ? h : 0)) * a.keep;
    char *base = static_cast<char *>(which ? a.v : a.k) + c;
    const bool weights = which == 0 && tid % vecs == 0 && col == 0, in = r0 < per;
    for (int j0 = 0; j0 < left; j0 += per * kBatch) {
        if (kept[min(j0 + per * kBatch, left) - 1] == min(j0 + per * kBatch, left) - 1) continue;  // (nothing moves yet)
        uint4 x[kBatch];
        float w[kBatch];
        int64_t dst[kBatch], wdst[kBatch];
#pragma unroll
        for (int e = 0; e < kBatch; ++e) {
            const int j = j0 + e * per + r0;
            dst[e] = -1;
            if (!in || j >= left) continue;
            const int i = kept[j];
            int64_t ps, pd;
            int rs, rd;
            if (i == j || !place(a, a.table, a.width, b, i, ps, rs) || !place(a, a.table, a.width, b, j, pd, rd)) continue;
            dst[e] = (pd * a.page_stride + rd * a.token_stride + h * a.head_stride) * a.esize;
            wdst[e] = pd * a.w_page + rd * a.w_token + h * a.w_head;
            x[e] = *reinterpret_cast<const uint4 *>(base + (ps * a.page_stride + rs * a.token_stride + h * a.head_stride) * a.esize);
            if (weights) w[e] = a.w[ps * a.w_page + rs * a.w_token + h * a.w_head];
        }
        __syncthreads();
#pragma unroll
        for (int e = 0; e < kBatch; ++e) {
            if (dst[e] < 0) continue;
            *reinterpret_cast<uint4 *>(base + dst[e]) = x[e];
            if (weights) a.w[wdst[e]] = w[e];
        }
        __syncthreads();
    }
    // keys that are appended behind the kept ones begin without a weight
    const int n = a.kv_lens[b];
    if (which || col || n > a.most) return;
    for (int i = left + tid; i < n; i += kMoveThreads) {
        int64_t page;
        int row;
        if (place(a, a.table, a.width, b, i, page, row)) a.w[page * a.w_page + row * a.w_token + h * a.w_head] = 0.f;
    }
}

}  // namespace

cudaError_t launch_evict_choose(const EvictArgs &a, cudaStream_t st) {
    static LaunchFit fit;
    const size_t most = sizeof(ChooseSmem) + (size_t)kHeld * 4;
    const cudaError_t e = fit.prepare(reinterpret_cast<const void *>(evict_choose_kernel), kThreads, most, nullptr);
    if (e != cudaSuccess) return e;
    // A cluster for each choice: as many CTAs as leave every SM one, while each has keys enough for its threads.
    const int64_t pairs = (int64_t)a.B * a.H, keys = a.most;
    int ranks = 1;
    while (ranks < 8 && pairs * ranks * 2 <= paged_sms() && keys > (int64_t)ranks * kThreads) ranks *= 2;
    const int room = (int)std::min<int64_t>(kHeld, (keys + ranks - 1) / ranks);
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = ranks;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cudaLaunchConfig_t c{};
    c.gridDim = dim3((unsigned)(pairs * ranks));
    c.blockDim = dim3(kThreads);
    c.dynamicSmemBytes = sizeof(ChooseSmem) + (size_t)room * 4;
    c.stream = st;
    c.attrs = &at;
    c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, evict_choose_kernel, a, room);
}

cudaError_t launch_evict_move(const EvictArgs &a, cudaStream_t st) {
    const int vecs = a.row_bytes / 16;
    if (a.out_table) {
        const int per = std::max(1, kMoveThreads / (2 * vecs));
        const int64_t blocks = std::min<int64_t>(((int64_t)a.keep * a.Hkv + per - 1) / per, 65535);
        for (int b0 = 0; b0 < a.B; b0 += 65535) {
            EvictArgs p = a;
            p.table += (int64_t)b0 * a.width;
            p.out_table += (int64_t)b0 * a.out_width;
            p.new_lens += b0;
            p.kept += (int64_t)b0 * a.H * a.keep;
            p.B = std::min(a.B - b0, 65535);
            evict_copy_kernel<<<dim3((unsigned)blocks, (unsigned)p.B), kMoveThreads, 0, st>>>(p);
        }
        return cudaGetLastError();
    }
    // columns of a row to CTAs of their own while there are SMs for them (32 bytes a row at least)
    int cols = 1;
    while (vecs % (cols * 2) == 0 && vecs / (cols * 2) >= 2 && (int64_t)a.B * a.Hkv * 2 * cols < 2 * paged_sms()) cols *= 2;
    evict_shift_kernel<<<(unsigned)((int64_t)a.B * a.Hkv * 2 * cols), kMoveThreads, 0, st>>>(a, cols);
    return cudaGetLastError();
}

}  // namespace ra

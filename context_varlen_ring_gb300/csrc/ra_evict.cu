// ra_evict.cu -- eviction from the paged cache: of a sequence's n keys the
// first `sinks`, the last `recent` and the heaviest of the rest stay, `keep`
// in all, in their order; their rows move to the front.
//
// Two kernels.  The choice is a search for the weight of the last key that
// stays, digit by digit over weights mapped to integers of the same order (11,
// 11 and 10 bits: a block's histogram of each digit in shared memory, the digit
// found in it by a sum from the top), and then two passes in which each warp
// counts, and then places, those of its keys that are above it and the first
// ones equal to it.  A long cache of few sequences is split over a cluster of
// CTAs, whose histograms are added through distributed shared memory.  It is a
// chain of barriers and loads that wait for one another, not bound by any rate
// (64 sequences of up to 8192 keys, 8 heads: 32 us; one of 65536: 23 us).  The
// move is a copy, bound by memory (1024 keys of each head: 84 us, 5.8 TB/s).
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

// The weights of keys i, i + STEP, ... (N of them, those below n; the others 0) of a choice: all loads of one kind
// together, so that a thread waits twice and not 2 N times.
template <int N, int STEP>
__device__ __forceinline__ void weight_keys(const EvictArgs &a, int b, int h, int i, int n, uint32_t (&x)[N]) {
    int page[N], row[N];
#pragma unroll
    for (int e = 0; e < N; ++e) {
        const int key = i + e * STEP, pi = a.page_shift >= 0 ? key >> a.page_shift : key / a.page_size;
        row[e] = key - pi * a.page_size;
        page[e] = key < n ? __ldg(a.table + b * a.width + pi) : 0;
    }
    float w[N];
    bool bad = false;
#pragma unroll
    for (int e = 0; e < N; ++e) {
        const bool in = i + e * STEP < n, fine = page[e] >= 0 && page[e] < a.n_pages;
        bad |= in && !fine;
        w[e] = 0.f;
        x[e] = in && fine;
        if (x[e]) w[e] = a.w[page[e] * a.w_page + row[e] * a.w_token + h * a.w_head];
    }
    if (a.H == 1)  // one choice for all heads, by their sum (h = 0)
        for (int j = 1; j < a.Hkv; ++j)
#pragma unroll
            for (int e = 0; e < N; ++e)
                if (x[e]) w[e] += a.w[page[e] * a.w_page + row[e] * a.w_token + j * a.w_head];
    if (bad) record_status(a.status, RA_ERR_DEVICE_BOUNDS);
#pragma unroll
    for (int e = 0; e < N; ++e) x[e] = x[e] ? ordered(w[e]) : 0;
}

struct ChooseSmem {
    alignas(16) int bins[3][kBins];  // of each digit
    int warp[32], digit[3], above[3];
    int gt[32], eq[32];              // each warp's keys above the threshold, and equal to it
    uint32_t held[1];                // (as many as the launch has room for)
};

template <bool CLUSTER>
__global__ void __launch_bounds__(CLUSTER ? 1024 : 512, CLUSTER ? 1 : 2) evict_choose_kernel(const EvictArgs a, int room) {
    constexpr int T = CLUSTER ? 1024 : 512, W = T / 32, PER = kBins / T;
    extern __shared__ __align__(16) uint8_t raw[];
    ChooseSmem &sm = *reinterpret_cast<ChooseSmem *>(raw);
    cg::cluster_group cluster = cg::this_cluster();
    const int ranks = CLUSTER ? (int)cluster.num_blocks() : 1, rank = CLUSTER ? (int)cluster.block_rank() : 0;
    auto sync = [&] {
        if (CLUSTER)
            cluster.sync();
        else
            __syncthreads();
    };
    auto other = [&](auto *p, int r) { return CLUSTER ? cluster.map_shared_rank(p, r) : p; };
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
    const int step = ranks * T, me = rank * T + tid;
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
    const int wh = a.H > 1 ? h : 0;
    auto key_at = [&](int i) {
        if (held) return sm.held[i];
        uint32_t x[1];
        weight_keys<1, T>(a, b, wh, at0 + i, at0 + cnt, x);
        return x[0];
    };
    for (int i = tid; i < 3 * kBins / 4; i += T) reinterpret_cast<int4 *>(sm.bins)[i] = make_int4(0, 0, 0, 0);
    if (held)
        for (int i = tid; i < cnt; i += 4 * T) {
            uint32_t x[4];
            weight_keys<4, T>(a, b, wh, at0 + i, at0 + cnt, x);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (i + e * T < cnt) sm.held[i + e * T] = x[e];
        }
    __syncthreads();
    // the threshold: its digits from the top, and how many of the keys above it are still wanted
    uint32_t prefix = 0, mask = 0;
    int need = want;
#pragma unroll 1
    for (int d = 0; d < 3; ++d) {
        const int shift = d == 0 ? 21 : d == 1 ? 10 : 0, bits = d == 2 ? 10 : 11;
        for (int i0 = 0; i0 < cnt; i0 += T) {
            const int i = i0 + tid;
            const uint32_t x = i < cnt ? key_at(i) : 0;
            const bool in = i < cnt && (x & mask) == prefix;
            const int digit = in ? (int)(x >> shift) & ((1 << bits) - 1) : -1;
            // lanes of one digit (weights of 0, mostly) are added at once
            int same;
            __match_all_sync(0xffffffffu, digit, &same);
            if (same) {
                if (lane == 0 && digit >= 0) atomicAdd(&sm.bins[d][digit], 32);
            } else if (digit >= 0) {
                atomicAdd(&sm.bins[d][digit], 1);
            }
        }
        sync();
        // PER bins a thread, the highest first: counts of the cluster, and their sum from the top
        int c[PER] = {}, mine = 0;
        const int top = kBins - PER - PER * tid;
#pragma unroll 4
        for (int r = 0; r < ranks; ++r) {
            const int *x = other(&sm.bins[d][0], r) + top;
#pragma unroll
            for (int e = 0; e < PER; e += 2) {
                const int2 y = *reinterpret_cast<const int2 *>(x + PER - 2 - e);
                c[e] += y.y;
                c[e + 1] += y.x;
            }
        }
#pragma unroll
        for (int e = 0; e < PER; ++e) mine += c[e];
        int sum = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += x;
        }
        if (lane == 31) sm.warp[warp] = sum;
        __syncthreads();
        int above = __reduce_add_sync(0xffffffffu, lane < warp ? sm.warp[lane] : 0) + sum - mine;
#pragma unroll
        for (int e = 0; e < PER; ++e) {
            if (above < need && above + c[e] >= need) {
                sm.above[d] = above;
                sm.digit[d] = top + PER - 1 - e;
            }
            above += c[e];
        }
        __syncthreads();
        need -= sm.above[d];
        prefix |= (uint32_t)sm.digit[d] << shift;
        mask |= (uint32_t)((1 << bits) - 1) << shift;
    }
    // each warp's keys (a run of them) above the threshold and equal to it; then those of the warps and CTAs ahead
    const int run = ((cnt + W - 1) / W + 31) & ~31, b0 = min(cnt, warp * run), b1 = min(cnt, b0 + run);
    int gt = 0, eq = 0;
    for (int i = b0 + lane; i < b1; i += 32) {
        const uint32_t x = key_at(i);
        gt += x > prefix;
        eq += x == prefix;
    }
    gt = __reduce_add_sync(0xffffffffu, gt);
    eq = __reduce_add_sync(0xffffffffu, eq);
    if (lane == 0) {
        sm.gt[warp] = gt;
        sm.eq[warp] = eq;
    }
    sync();
    gt = lane < warp ? sm.gt[lane] : 0;
    eq = lane < warp ? sm.eq[lane] : 0;
    if (CLUSTER && lane < W)
        for (int r = 0; r < rank; ++r) {
            gt += *(other(&sm.gt[0], r) + lane);
            eq += *(other(&sm.eq[0], r) + lane);
        }
    gt = __reduce_add_sync(0xffffffffu, gt);
    eq = __reduce_add_sync(0xffffffffu, eq);
    // of the equal ones, the first `need` stay: a key's place is the count of those above ahead of it, and of the equal
    // ones ahead of it as far as they stay
    for (int i0 = b0; i0 < b1; i0 += 32) {
        const int i = i0 + lane;
        const uint32_t x = i < b1 ? key_at(i) : 0;
        const bool g = i < b1 && x > prefix, e = i < b1 && x == prefix;
        const uint32_t bg = __ballot_sync(0xffffffffu, g), be = __ballot_sync(0xffffffffu, e), below = (1u << lane) - 1;
        const int ga = gt + __popc(bg & below), ea = eq + __popc(be & below);
        if (g || (e && ea < need)) kept[first + ga + min(ea, need)] = at0 + i;
        gt += __popc(bg);
        eq += __popc(be);
    }
    if (CLUSTER) cluster.sync();  // (no CTA ends while another reads its counts)
}

// ------------------------------------------------------------ the move
constexpr int kMoveThreads = 256;

// The move's blocks are set up while the choice ends (they wait for it before they read anything of it).
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
template <typename... P, typename... A>
cudaError_t launch_next(void (*kernel)(P...), dim3 grid, cudaStream_t st, A... args) {
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t c{};
    c.gridDim = grid;
    c.blockDim = dim3(kMoveThreads);
    c.stream = st;
    c.attrs = &at;
    c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, kernel, args...);
}

// To other pages: a warp takes ROWS rows of one head, looks up a row's places in each lane, and then copies them 16 bytes
// a lane, kCopies pieces a lane on their way at once (8 of them, in 78 registers: 121 us for 64 sequences of 8 heads and 1024 keys
// kept; five blocks an SM with 4: 90).
constexpr int kCopies = 4;
template <int ROWS>
__global__ void __launch_bounds__(kMoveThreads, 5) evict_copy_kernel(const EvictArgs a) {
    const int b = blockIdx.y, lane = threadIdx.x & 31;
    pdl_wait();
    const int left = a.new_lens[b], vecs = a.row_bytes / 16, pieces = 2 * vecs;  // of a row: K, then V
    const int64_t blocks = (int64_t)((left + ROWS - 1) / ROWS) * a.Hkv;
    const int64_t off_v = static_cast<char *>(a.v) - static_cast<char *>(a.k);
    for (int64_t u = blockIdx.x * (kMoveThreads / 32) + (threadIdx.x >> 5); u < blocks; u += (int64_t)gridDim.x * (kMoveThreads / 32)) {
        const int j0 = (int)(u / a.Hkv) * ROWS, h = (int)(u % a.Hkv), j = j0 + lane, rows = min(ROWS, left - j0);
        int64_t src = -1, dst = -1;  // bytes from the start of K
        if (lane < rows) {
            const int i = __ldg(a.kept + ((int64_t)b * a.H + (a.H > 1 ? h : 0)) * a.keep + j);
            int64_t ps, pd;
            int rs, rd;
            const bool from = place(a, a.table, a.width, b, i, ps, rs), to = place(a, a.out_table, a.out_width, b, j, pd, rd);
            if (from && to) {
                src = (ps * a.page_stride + rs * a.token_stride + h * a.head_stride) * a.esize;
                dst = (pd * a.page_stride + rd * a.token_stride + h * a.head_stride) * a.esize;
                a.w[pd * a.w_page + rd * a.w_token + h * a.w_head] = a.w[ps * a.w_page + rs * a.w_token + h * a.w_head];
            }
        }
        int row = lane / pieces, piece = lane - row * pieces;
        const int hop = 32 / pieces, rest = 32 - hop * pieces;  // rows and pieces that 32 lanes go on by
        const int steps = (rows * pieces + 31) / 32;
        for (int s0 = 0; s0 < steps; s0 += kCopies) {
            uint4 x[kCopies];
            char *to[kCopies];
#pragma unroll
            for (int e = 0; e < kCopies; ++e) {
                const int r = min(row, 31);
                const int64_t f = __shfl_sync(0xffffffffu, src, r), d = __shfl_sync(0xffffffffu, dst, r);
                const int64_t c = piece * 16 + (piece >= vecs ? off_v - (int64_t)vecs * 16 : 0);
                to[e] = row < rows && f >= 0 ? static_cast<char *>(a.k) + d + c : nullptr;
                if (to[e]) x[e] = __ldcs(reinterpret_cast<const uint4 *>(static_cast<char *>(a.k) + f + c));
                row += hop;
                piece += rest;
                if (piece >= pieces) {
                    piece -= pieces;
                    ++row;
                }
            }
#pragma unroll
            for (int e = 0; e < kCopies; ++e)
                if (to[e]) __stcs(reinterpret_cast<uint4 *>(to[e]), x[e]);
        }
    }
}

// In place: kept key j comes from a place at or behind j, and places only grow, so a batch of rows may be written once
// all of it is read: every row that it overwrites was read in this batch or before.  A CTA walks one head's batches for
// some columns of K or of V (64 sequences of up to 8192 keys to 1024 of each of 8 heads, choice and all: 234 us; one of
// 65536 to 4096: 83).
constexpr int kBatch = 8;  // 16-byte pieces a thread
__global__ void __launch_bounds__(kMoveThreads) evict_shift_kernel(const EvictArgs a, int cols) {
    const int vecs = a.row_bytes / 16 / cols;  // pieces of a row that this CTA moves
    const int col = blockIdx.x % cols, which = blockIdx.x / cols % 2, pair = blockIdx.x / (2 * cols);
    const int b = pair / a.Hkv, h = pair % a.Hkv;
    pdl_wait();
    const int left = a.new_lens[b];
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
    static LaunchFit fit[2];
    const size_t most = sizeof(ChooseSmem) + (size_t)kHeld * 4;
    // A cluster for each choice: as many CTAs as leave every SM one, while each has keys enough for its threads.
    const int64_t pairs = (int64_t)a.B * a.H, keys = a.most;
    int ranks = 1;
    while (ranks < 8 && pairs * ranks * 2 <= paged_sms() && keys > (int64_t)ranks * 1024) ranks *= 2;
    auto kernel = ranks > 1 ? evict_choose_kernel<true> : evict_choose_kernel<false>;
    const cudaError_t e = fit[ranks > 1].prepare(reinterpret_cast<const void *>(kernel), ranks > 1 ? 1024 : 512, most, nullptr);
    if (e != cudaSuccess) return e;
    const int room = (int)std::min<int64_t>(kHeld, (keys + ranks - 1) / ranks);
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = ranks;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cudaLaunchConfig_t c{};
    c.gridDim = dim3((unsigned)(pairs * ranks));
    c.blockDim = dim3(ranks > 1 ? 1024 : 512);
    c.dynamicSmemBytes = sizeof(ChooseSmem) + (size_t)room * 4;
    c.stream = st;
    c.attrs = &at;
    c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, kernel, a, room);
}

cudaError_t launch_evict_move(const EvictArgs &a, cudaStream_t st) {
    if (a.out_table) {
        // (few rows: more warps, each with fewer)
        const bool few = (int64_t)a.B * a.Hkv * a.keep < (int64_t)paged_sms() * 16 * 32;
        const int rows = few ? 8 : 32;
        const int64_t warps = ((int64_t)a.keep + rows - 1) / rows * a.Hkv;
        const int64_t blocks = std::min<int64_t>((warps + kMoveThreads / 32 - 1) / (kMoveThreads / 32), 65535);
        for (int b0 = 0; b0 < a.B; b0 += 65535) {
            EvictArgs p = a;
            p.table += (int64_t)b0 * a.width;
            p.out_table += (int64_t)b0 * a.out_width;
            p.new_lens += b0;
            p.kept += (int64_t)b0 * a.H * a.keep;
            p.B = std::min(a.B - b0, 65535);
            const cudaError_t e = launch_next(few ? evict_copy_kernel<8> : evict_copy_kernel<32>, dim3((unsigned)blocks, (unsigned)p.B), st, p);
            if (e != cudaSuccess) return e;
        }
        return cudaSuccess;
    }
    // Columns of a row to CTAs of their own while there are SMs for them (32 bytes a row at least): one of 65536 keys to
    // 4096, 8 heads, 83 us, by whole rows 220; 3 of 3000 to 700, 4 heads, 24 and 47; 16 of 9000 to 2048, 8 heads, where
    // rows are cut in two, 171 and 162.
    const int vecs = a.row_bytes / 16;
    int cols = 1;
    while (vecs % (cols * 2) == 0 && vecs / (cols * 2) >= 2 && (int64_t)a.B * a.Hkv * 2 * cols < 2 * paged_sms()) cols *= 2;
    return launch_next(evict_shift_kernel, dim3((unsigned)((int64_t)a.B * a.Hkv * 2 * cols)), st, a, cols);
}

}  // namespace ra

// ra_weights_tc.cu -- key weights of many query rows (bf16, d = 128) on the
// 5th-generation tensor cores: chunks of a prompt, and prefixes of a batch.
//
// Bound: 2 d flops and one exponential for each (row, key) pair; the tensor
// pipe and the special-function unit take 512 cycles each for 128 x 128 of them
// (2048 tokens of 32 heads behind 30720 keys of 8: 420 us, 1.27 PFLOP/s).
// Keys are the rows of S (A operand, a key a TMEM lane) and query rows its
// columns, so a key's weight is summed in one thread's registers and no sum
// passes between threads but one of each unit.  A unit is 256 keys of one KV head:
// two tiles in shared memory that meet every tile of 128 query rows, which come by
// TMA through a ring.  Each tile of keys has two buffers of S and two warpgroups,
// which take its tiles of rows in turn, so that the next product runs beside the
// exponentials (a warpgroup with half of every tile's columns waits twice as
// often: 439 us).  One more warp makes the rows' offsets.  The next unit's keys are
// loaded beside this unit's rows.  Every wait is bounded as in the rest of the
// library.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstring>

#include "ra_internal.h"
#include "ra_serve.cuh"
#include "ra_weights.cuh"

namespace ra {
namespace {

using namespace weights;

constexpr int kThreads = 640;
constexpr int kKeys = 256;             // of a unit
constexpr uint32_t kHalf = 16384;      // 128 rows x 128 B (64 bf16), 128-byte swizzle
constexpr uint32_t kTile = 2 * kHalf;  // 128 rows x 128 bf16
constexpr int kRing = 4;               // tiles of rows
constexpr uint32_t kOffQ = 2 * kTile;  // behind the keys
constexpr uint32_t kOffBar = kOffQ + kRing * kTile;
constexpr uint32_t kSmem = kOffBar + 384 + 1024;

constexpr int kPlaces = 8;

struct TcParams {
    CUtensorMap tmQ, tmK;
    WeightArgs a;
    int box, log2G, rows_inner;  // as in the paged attention's tensor maps
    unsigned long long budget_ns;
};

struct Shared {
    Line line;
    alignas(16) float off[kRing][128];  // (read as float4) of the rows of a tile: -lse in base 2
    int none[kRing];                    // whether any of a tile's rows adds nothing
    float sum[2][kPlaces][128];         // of the odd tiles of rows, a unit after another
};

struct Unit {
    Segment g;
    int s, h, k0, first, tiles, parts;  // first row; tiles of 128 rows; tiles of 128 keys
    bool own;
};

__global__ void __launch_bounds__(kThreads, 1) weights_tc_kernel(const __grid_constant__ TcParams p) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ Shared sh;
    const WeightArgs &a = p.a;
    const uint32_t raw_s = smem_u32(smem_raw), base_s = (raw_s + 1023u) & ~1023u;
    uint8_t *base = smem_raw + (base_s - raw_s);
    uint64_t *bars = reinterpret_cast<uint64_t *>(base + kOffBar);
    uint64_t *k_full = bars + 0;    // a unit's keys landed
    uint64_t *k_empty = bars + 1;
    uint64_t *q_full = bars + 2;    // [kRing] a tile of rows
    uint64_t *q_empty = bars + 6;   // [kRing]
    uint64_t *s_full = bars + 10;   // [2][2] S of a warpgroup's buffer
    uint64_t *s_empty = bars + 14;  // [2][2] (128 arrivals)
    uint64_t *part = bars + 18;     // [2][kPlaces] a unit's odd tiles are summed (128 arrivals)
    uint64_t *mma_done = bars + 34;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 35);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(bars + 36);
    uint64_t *o_full = bars + 37;   // [kRing] a tile's offsets
    uint64_t *o_empty = bars + 41;  // [kRing] (8 warps)
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        *abort_flag = 0;
        mbar_init(k_full, 1);
        mbar_init(k_empty, 1);
        for (int i = 0; i < kRing; ++i) {
            mbar_init(q_full + i, 1);
            mbar_init(q_empty + i, 1);
            mbar_init(o_full + i, 1);
            mbar_init(o_empty + i, 8);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(s_full + i, 1);
            mbar_init(s_empty + i, 128);
        }
        for (int i = 0; i < 2 * kPlaces; ++i) mbar_init(part + i, 128);
        mbar_init(mma_done, 1);
        fence_mbar_init();
        tma_prefetch_desc(&p.tmQ);
        tma_prefetch_desc(&p.tmK);
    }
    // (256 of the threads line the segments up: kSegs is a multiple of 256)
    const int tiles = line_up<256, kThreads>(a, 0, 8, sh.line);
    if (tiles < 0) {
        if (threadIdx.x == 0) record_status(a.status, RA_ERR_DEVICE_BOUNDS);
        return;
    }
    if (warp == 2) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const WaitCtl wc{abort_flag, a.status, p.budget_ns};
    const int64_t units = (int64_t)tiles * a.Hkv;
    auto unit = [&](int64_t u, Unit &w) {
        const int tile = (int)(u / a.Hkv);
        w.h = (int)(u - (int64_t)tile * a.Hkv);
        w.s = find(sh.line, tile);
        w.k0 = (tile - sh.line.at[w.s]) * kKeys;
        segment(a, w.s, w.g);
        w.own = w.s < a.B;
        const int rows = w.g.n << p.log2G;
        w.first = w.own && a.causal ? (max(0, w.k0 - (w.g.len - w.g.n)) << p.log2G) & ~127 : 0;
        w.tiles = (rows - w.first + 127) / 128;
        w.parts = w.g.len - w.k0 > 128 ? 2 : 1;
    };

    if (warp == 0) {
        // ------------------------------------------------ loads
        uint32_t nk = 0, nq = 0;
        bool ok = true;
        const uint64_t policy = l2_evict_first();
        const int boxes = 256 / p.box;  // of a tile: 128 / box row ranges x 2 halves of d
        for (int64_t u = blockIdx.x; u < units && ok; u += gridDim.x) {
            Unit w;
            unit(u, w);
            ok = mbar_wait_warp(k_empty, (nk & 1u) ^ 1u, wc);
            if (!ok) break;
            if (lane == 0) mbar_arrive_expect_tx(k_full, w.parts * kTile);
            __syncwarp();
            ++nk;
            for (int t = 0; t < w.parts; ++t) {
                if (lane < boxes) {
                    const int key = w.k0 + t * 128 + (lane >> 1) * p.box;
                    const int pi = a.page_shift >= 0 ? key >> a.page_shift : key / a.page_size, row = key - pi * a.page_size;
                    int page = (int)a.n_pages;  // (outside the cache: filled with zeros)
                    if (key < w.g.len) {
                        const int f = w.s >= a.B;
                        page = __ldg(a.table[f] + (int64_t)(w.s - (f ? a.B : 0)) * a.width[f] + pi);
                        if (page < 0 || page >= a.n_pages) {
                            record_status(a.status, RA_ERR_DEVICE_BOUNDS);
                            page = (int)a.n_pages;
                        }
                    }
                    const int c1 = p.rows_inner ? row : w.h, c2 = p.rows_inner ? w.h : row;
                    tma_load_4d_hint(base + t * kTile + (lane & 1) * kHalf + (lane >> 1) * p.box * 128, &p.tmK,
                                     k_full, (lane & 1) * 64, c1, c2, page, policy);
                }
                __syncwarp();
            }
            for (int j = 0; j < w.tiles && ok; ++j, ++nq) {
                const uint32_t s = nq % kRing;
                ok = mbar_wait_warp(q_empty + s, ((nq / kRing) & 1u) ^ 1u, wc);
                if (!ok) break;
                if (lane == 0) {
                    const int tok = w.g.tok0 + ((w.first + j * 128) >> p.log2G), hq = w.h << p.log2G;
                    mbar_arrive_expect_tx(q_full + s, kTile);
                    tma_load_3d(base + kOffQ + s * kTile, &p.tmQ, q_full + s, 0, hq, tok);
                    tma_load_3d(base + kOffQ + s * kTile + kHalf, &p.tmQ, q_full + s, 64, hq, tok);
                }
                __syncwarp();
            }
        }
        if (lane == 0) {
            // the last copies must have landed before the CTA may exit
            volatile int local_abort = 0;
            const WaitCtl drain{&local_abort, a.status, p.budget_ns};
            if (nk > 0) (void)mbar_wait(k_full, (nk - 1) & 1u, drain);
            for (uint32_t i = nq > kRing ? nq - kRing : 0; i < nq; ++i) (void)mbar_wait(q_full + i % kRing, (i / kRing) & 1u, drain);
        }
    } else if (warp == 1) {
        // ------------------------------------------------ products
        const uint32_t idesc = idesc_bf16_f32(128, 128, 0, 0);
        uint32_t nk = 0, nq = 0, ns[2][2] = {};  // (uses of each buffer)
        bool ok = true;
        for (int64_t u = blockIdx.x; u < units && ok; u += gridDim.x) {
            Unit w;
            unit(u, w);
            ok = mbar_wait_warp(k_full, nk & 1u, wc);
            ++nk;
            for (int j = 0; j < w.tiles && ok; ++j, ++nq) {
                const uint32_t s = nq % kRing, b = nq & 1;
                ok = mbar_wait_warp(q_full + s, (nq / kRing) & 1u, wc);
                if (!ok) break;
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    if (t >= w.parts) break;
                    ok = mbar_wait_warp(s_empty + 2 * t + b, ((b ? ns[t][1] : ns[t][0]) & 1u) ^ 1u, wc);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t dk = sdesc_sw128(base_s + t * kTile, 16, 1024);
                    const uint64_t dq = sdesc_sw128(base_s + kOffQ + s * kTile, 16, 1024);
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks) {
                        const uint32_t o = ((uint32_t)(ks >> 2) * kHalf + (uint32_t)(ks & 3) * 32u) >> 4;
                        tc_mma_ss_w(tmem + 256u * t + 128u * b, dk + o, dq + o, idesc, ks > 0);
                    }
                    tc_commit_w(s_full + 2 * t + b);
                    ns[t][0] += b == 0;
                    ns[t][1] += b;
                }
                tc_commit_w(q_empty + s);
            }
            tc_commit_w(k_empty);
        }
        // every product issued must have completed before TMEM is released
        tc_commit_w(mma_done);
        volatile int local_abort = 0;
        const WaitCtl drain{&local_abort, a.status, p.budget_ns};
        (void)mbar_wait_warp(mma_done, 0, drain);
    } else if (warp == 3) {
        // ------------------------------------------------ the rows' offsets, four a lane, for all of the warps below
        // (2048 tokens at 32768 keys; each for itself, 488 us: 452 so)
        uint32_t no = 0;
        bool ok = true;
        for (int64_t u = blockIdx.x; u < units && ok; u += gridDim.x) {
            Unit w;
            unit(u, w);
            const int rows = w.g.n << p.log2G;
            for (int j = 0; j < w.tiles; ++j, ++no) {
                const int r0 = w.first + 128 * j + 4 * lane;
                float x[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int r = r0 + e < rows ? r0 + e : 0;
                    x[e] = __ldg(a.lse + (int64_t)(w.h * a.G + (r & (a.G - 1))) * a.T + w.g.tok0 + (r >> p.log2G));
                }
                ok = mbar_wait_warp(o_empty + no % kRing, ((no / kRing) & 1u) ^ 1u, wc);
                if (!ok) break;
                bool any = false;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const bool none = r0 + e >= rows || x[e] == -INFINITY;
                    x[e] = none ? -INFINITY : -x[e] * 1.4426950408889634f;
                    any |= x[e] == -INFINITY;
                }
                const uint32_t vote = __ballot_sync(0xffffffffu, any);
                *reinterpret_cast<float4 *>(sh.off[no % kRing] + 4 * lane) = make_float4(x[0], x[1], x[2], x[3]);
                if (lane == 0) sh.none[no % kRing] = vote != 0;
                __syncwarp();
                if (lane == 0) mbar_arrive(o_full + no % kRing);
            }
        }
    } else if (warp >= 4) {
        // ------------------------------------------------ exponentials and sums
        // two warpgroups a tile of keys, which take its tiles of rows in turn
        const int k = warp >= 12 ? 1 : 0;
        const uint32_t b = (warp >> 2) & 1 ? 0 : 1;  // its buffer: warps 4 .. 7 and 12 .. 15 have the even tiles
        const int m = (warp & 3) * 32 + lane;        // TMEM lane: the key
        const uint32_t tS = tmem + ((uint32_t)((warp & 3) * 32) << 16) + 256u * k + 128u * b;
        uint32_t ns = 0, nu = 0, no = 0;
        bool ok = true;
        for (int64_t u = blockIdx.x; u < units && ok; u += gridDim.x) {
            Unit w;
            unit(u, w);
            if (k >= w.parts) {
                for (int j = 0; j < w.tiles && ok; ++j, ++no) {
                    if ((no & 1) != b) continue;
                    ok = mbar_wait_warp(o_full + no % kRing, (no / kRing) & 1u, wc);
                    if (ok && lane == 0) mbar_arrive(o_empty + no % kRing);
                }
                continue;
            }
            const int key = w.k0 + 128 * k + m;
            // the first row that sees the key, and the first that all of the warp's keys are seen by (a key far ahead of the
            // new tokens, which 32 bits do not hold times the heads, is seen by all; one behind the end is not written)
            const int token = w.own && a.causal ? key - (w.g.len - w.g.n) : 0, last = w.own && a.causal ? token + 31 - lane : 0;
            const int from = min(max(token, 0), w.g.n) * a.G, all_from = min(max(last, 0), w.g.n) * a.G;
            float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
            const float2 sl2 = make_float2(a.scale_log2, a.scale_log2);
#pragma unroll 1
            for (int j = 0; j < w.tiles; ++j, ++no) {
                if ((no & 1) != b) continue;
                const uint32_t slot = no % kRing, ph = ns++ & 1;
                const int r0 = w.first + 128 * j;
                // (both looked at in one go: they are there as a rule)
                const bool o = mbar_try_wait(o_full + slot, (no / kRing) & 1u), s = mbar_try_wait(s_full + 2 * k + b, ph);
                if (!__all_sync(0xffffffffu, o && s)) {
                    ok = mbar_wait_warp(o_full + slot, (no / kRing) & 1u, wc) && mbar_wait_warp(s_full + 2 * k + b, ph, wc);
                    if (!ok) break;
                }
                tc_fence_after();
                const bool cut = sh.none[slot] || all_from > r0;
#pragma unroll
                for (int c = 0; c < 128; c += 32) {
                    uint32_t v[32];
                    tmem_ld32(tS + c, v);
                    if (c == 96) {  // (all columns are read)
                        tc_fence_before();
                        mbar_arrive(s_empty + 2 * k + b);
                    }
                    const float4 *off = reinterpret_cast<const float4 *>(sh.off[slot] + c);
                    if (!cut) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float4 f = off[i];
                            const float2 x = fma2(make_float2(__uint_as_float(v[4 * i]), __uint_as_float(v[4 * i + 1])), sl2, make_float2(f.x, f.y));
                            const float2 y = fma2(make_float2(__uint_as_float(v[4 * i + 2]), __uint_as_float(v[4 * i + 3])), sl2, make_float2(f.z, f.w));
                            sum[0] = add2(sum[0], make_float2(ex2_approx(x.x), ex2_approx(x.y)));
                            sum[1] = add2(sum[1], make_float2(ex2_approx(y.x), ex2_approx(y.y)));
                        }
                    } else {  // rows that do not see the key, or add nothing (their scores may be anything)
                        const int seen = from - r0 - c;
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            const float f = sh.off[slot][c + i];
                            const float x = ex2_approx(fmaf(__uint_as_float(v[i]), a.scale_log2, f));
                            sum[0].x += i >= seen && f != -INFINITY ? x : 0.f;
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(o_empty + slot);
            }
            // the odd tiles' sums go to the threads of the even ones.  Products are issued tile after tile, and a tile's
            // only when its buffer was read: so the odd ones are two tiles ahead at most, and, with units of one tile,
            // where every other one is nothing to them, four units: of the eight places none is written before it was read
            const float all = (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
            const uint32_t at = nu % kPlaces;
            if (b) {
                sh.sum[k][at][m] = all;
                mbar_arrive(part + kPlaces * k + at);
            } else {
                ok = ok && mbar_wait_warp(part + kPlaces * k + at, (nu / kPlaces) & 1u, wc);
                int64_t page;
                int row;
                if (ok && key < w.g.len && place(a, w.s, key, page, row))
                    a.w[page * a.w_page + row * a.w_token + w.h * a.w_head] += all + sh.sum[k][at][m];
            }
            ++nu;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 2) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

}  // namespace

bool weights_tc_maps(const WeightArgs &a, PagedMaps &m) {
    PagedArgs p{};  // (the paged attention's maps of q and of the cache)
    p.q = a.q;
    p.q_stride = a.q_stride;
    p.T = a.T;
    p.Hq = a.Hq;
    p.Hkv = a.Hkv;
    p.G = a.G;
    p.d = a.d;
    p.dtype = a.dtype;
    p.k = p.v = a.k;
    p.n_pages = a.n_pages;
    p.page_stride = a.page_stride;
    p.token_stride = a.token_stride;
    p.head_stride = a.head_stride;
    p.page_size = a.page_size;
    p.scale_log2 = 1.f;
    return a.B + a.n_groups <= kSegs && paged_tc_maps(p, m);
}

cudaError_t launch_weights_tc(const WeightArgs &a, const PagedMaps &m, cudaStream_t st) {
    TcParams p;
    memset(&p, 0, sizeof(p));
    p.tmQ = m.q;
    p.tmK = m.k;
    p.rows_inner = m.rows_inner;
    p.a = a;
    p.box = a.page_size < 128 ? a.page_size : 128;
    while ((1 << p.log2G) < a.G) ++p.log2G;
    p.budget_ns = wait_budget_ns();
    static LaunchFit fit;
    static_assert(kSmem + sizeof(Shared) <= 232448, "shared memory of one CTA");
    const cudaError_t e = fit.prepare(reinterpret_cast<const void *>(weights_tc_kernel), kThreads, kSmem, nullptr);
    if (e != cudaSuccess) return e;
    weights_tc_kernel<<<paged_sms(), kThreads, kSmem, st>>>(p);
    return cudaGetLastError();
}

}  // namespace ra

// ra_paged_tc.cu -- paged attention for many query rows per KV head (bf16,
// d = 128) on the 5th-generation tensor cores: a prefix that a batch shares,
// and sequences with several query tokens.
//
// Mathematics and bound: R rows (query tokens x the G query heads of one KV
// head) against n keys take 4 d R n flops and read 4 d n bytes of keys, so
// above about 280 rows the tensor rate bounds it, below that memory.
//
// Design, next to tc_fwd_kernel of the packed ring (same products, same
// softmax): persistent CTAs of 12 warps, one a SM, each with an equal run of
// the line of key tiles (so no claims and no descriptor ring: every role
// walks the same run by itself).  A unit has up to 256 rows.
//  * 129 to 256 rows: two tiles of 128 rows share each K and V tile; softmax
//    group k (4 warps, a thread a row) owns row tile k.
//  * up to 128 rows: both softmax groups own the same rows and take alternate
//    key tiles, with a partial each, so one group's softmax hides behind the
//    other's products although there is only one tile of rows.
// Pages: a 4-D tensor map (d, head, row in page, page; head and row in the
// order of their strides) with a box of min(page, 128) rows; the lanes of the
// producer warp look up a page each and issue the boxes of a tile side by side.
// Keys behind the length come from a page outside the cache, which TMA fills
// with zeros; what a last page holds behind the length is masked in S, and its V
// rows are zeroed in shared memory before the product, so it may be anything.
// Measured: a prefix of 65536 keys for 128 requests of 64 heads (8 of keys) in
// 0.76 of the measured bf16 rate: a step of 128 keys takes 3130 cycles for 2048
// of products, of which a row tile's softmax 1720, its P V and next S the rest.
// Every wait is bounded as in the rest of the library.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <mutex>

#include "ra_dev.cuh"
#include "ra_internal.h"
#include "ra_kernels.h"
#include "ra_paged.cuh"

namespace ra {
namespace {

using namespace dev;

constexpr int kThreads = 384;
constexpr int kSlots = 5;
constexpr uint32_t kHalf = 16384;      // 128 rows x 128 B (64 bf16), 128-byte swizzle
constexpr uint32_t kTile = 2 * kHalf;  // 128 rows x 128 bf16
constexpr uint32_t kOffKV = 2 * kTile;
constexpr uint32_t kOffBar = kOffKV + kSlots * kTile;
constexpr uint32_t kSmem = kOffBar + 256 + 1024;  // + barriers + alignment slack

struct TcParams {
    CUtensorMap tmQ, tmK, tmV;
    PagedArgs a;
    int fi, late, box, log2G;  // family, whether it waits last, rows a box
    int rows_inner;      // the maps' dimensions: (d, row in page, head, page) instead of (d, head, row in page, page)
    unsigned long long budget_ns;
};

// What one CTA does of one unit: steps of one key tile (two row tiles) or of
// two key tiles (one row tile).
struct Walk {
    PagedUnit u;
    bool pair;  // two row tiles
    int tend;   // key tiles [u.t0, tend): those that any row sees
};

// Bits [0, n) of the 32 columns starting at `base`.
__device__ __forceinline__ uint32_t low_bits(int n, int base) {
    const int k = min(max(n - base, 0), 32);
    return k == 32 ? 0xffffffffu : (1u << k) - 1u;
}

// Columns of a tile that the softmax holds at once, in rolled loops: the
// kernel's short runs wait for instructions as much as for anything (with the
// tile unrolled the first one took 10000 to 17000 cycles, a later one 3400).
constexpr int kCols = 64, kChunks = 128 / kCols;  // (the loads and stores below are of 64 and 32 columns)
__device__ __forceinline__ void mask_cols(uint32_t (&v)[kCols], int seen, int base) {
#pragma unroll
    for (int c = 0; c < kCols; c += 32) {
        const uint32_t bits = low_bits(seen, base + c);
#pragma unroll
        for (int i = 0; i < 32; ++i) v[c + i] = ((bits >> i) & 1u) ? v[c + i] : 0xff800000u;  // -inf
    }
}

// A descriptor `bytes` further on: its address field is the low word's, and
// no address of shared memory leaves it.
__device__ __forceinline__ uint64_t desc_at(uint64_t d, uint32_t bytes) { return d + (bytes >> 4); }
__device__ __forceinline__ void issue_s(uint32_t d_tmem, uint64_t q, uint64_t k, uint32_t idesc) {
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) {
        const uint32_t off = (uint32_t)(ks >> 2) * kHalf + (uint32_t)(ks & 3) * 32u;
        tc_mma_ss_w(d_tmem, desc_at(q, off), desc_at(k, off), idesc, ks > 0);
    }
}
__device__ __forceinline__ void issue_pv(uint32_t d_tmem, uint32_t p_tmem, uint64_t v, uint32_t idesc,
                                         uint32_t accumulate) {
#pragma unroll
    for (int ks = 0; ks < 8; ++ks)
        tc_mma_ts_w(d_tmem, p_tmem + 8u * ks, desc_at(v, (uint32_t)ks * 2048u), idesc,
                    (accumulate || ks > 0) ? 1u : 0u);
}

__global__ void __launch_bounds__(kThreads, 1) paged_tc_kernel(const __grid_constant__ TcParams p) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_s = smem_u32(smem_raw);
    const uint32_t base_s = (raw_s + 1023u) & ~1023u;
    uint8_t *base = smem_raw + (base_s - raw_s);
    uint64_t *bars = reinterpret_cast<uint64_t *>(base + kOffBar);
    uint64_t *q_full = bars + 0;     // Q tiles of a unit landed (one phase per unit)
    uint64_t *q_empty = bars + 1;    // the unit's last S products are done with Q
    uint64_t *kv_full = bars + 2;    // [kSlots]
    uint64_t *kv_empty = bars + 7;   // [kSlots]
    uint64_t *s_full = bars + 12;    // [2] S of a group computed
    uint64_t *p_ready = bars + 14;   // [2] P of a group written to TMEM (128 arrivals)
    uint64_t *o_done = bars + 16;    // [2] a group's PVs of a unit done
    uint64_t *mma_done = bars + 18;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 19);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(bars + 20);
    const PagedArgs &a = p.a;
    const PagedFamily &f = a.f[p.fi];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        *abort_flag = 0;
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(kv_full + i, 1);
            mbar_init(kv_empty + i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(s_full + i, 1);
            mbar_init(p_ready + i, 128);
            mbar_init(o_done + i, 1);
        }
        mbar_init(mma_done, 1);
        fence_mbar_init();
        tma_prefetch_desc(&p.tmQ);
        tma_prefetch_desc(&p.tmK);
        tma_prefetch_desc(&p.tmV);
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

    // Each warp's place in the CTA's run: in shared memory, so that it holds no
    // registers in the loops over key tiles.
    __shared__ PagedWalk place[kThreads / 32];
    __shared__ PlanShared plan;
    if (warp < 4) {
        if (!p.late) pdl_wait();
        pdl_launch();
        const PagedWalk k = paged_begin<128, 1>(a, f, p.fi, plan);
        if (lane == 0) {
            place[warp] = k;
            place[warp + 4] = k;
            place[warp + 8] = k;
        }
        __syncwarp();
        asm volatile("bar.arrive 2, 384;" ::: "memory");  // the softmax warps read theirs
    }
    // The CTA's units in order, the same for every role.
    auto next_unit = [&](Walk &w) {
        PagedWalk k = place[warp];
        __syncwarp();
        if (!paged_unit(a, f, p.fi, k, w.u)) return false;
        if (lane == 0) place[warp] = k;
        __syncwarp();
        w.pair = w.u.rows > 128;
        const int sees = paged_limit(a, w.u, p.fi, w.u.r0 + w.u.rows - 1);
        w.tend = min(w.u.t1, max(w.u.t0, (sees + 127) / 128));
        return true;
    };

    // Registers: 128 x 80 + 256 x 200 = 61440, within the 384 x 168 = 64512 of the launch.
    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 80;\n" ::: "memory");
        if (warp == 0) {
            // -------------------------------------------- producer
            uint32_t n = 0;  // K and V tiles loaded
            int nq = 0, ok = 1;
            const uint64_t policy = l2_evict_first();
            const int boxes = 256 / p.box;  // of a tile: 128 / box row ranges x 2 halves of d
            for (Walk w; ok && next_unit(w);) {
                const int tok = w.u.tok0 + (w.u.r0 >> p.log2G), hq = w.u.h << p.log2G;
                // the page of this lane's box of a tile, as the table has it (n_pages: outside the cache, filled with zeros)
                auto look_up = [&](int t) {
                    const int key = t * 128 + (lane >> 1) * p.box;
                    return lane < boxes && key < w.u.len ? __ldg(f.table + (int64_t)w.u.s * f.width + paged_page(a, key))
                                                         : (int)a.n_pages;
                };
                int pa = look_up(w.u.t0), pb = look_up(w.u.t0 + 1);
                if (lane == 0) {
                    if (nq > 0) ok = mbar_wait(q_empty, (nq - 1) & 1u, wc);
                    if (ok) {
                        mbar_arrive_expect_tx(q_full, (w.pair ? 2u : 1u) * kTile);
                        for (int k = 0; k < (w.pair ? 2 : 1); ++k) {
                            tma_load_3d(base + k * kTile, &p.tmQ, q_full, 0, hq, tok + k * (128 >> p.log2G));
                            tma_load_3d(base + k * kTile + kHalf, &p.tmQ, q_full, 64, hq, tok + k * (128 >> p.log2G));
                        }
                        ++nq;
                    }
                }
                ok = __shfl_sync(0xffffffffu, ok, 0);
                auto load = [&](const CUtensorMap *m, int t, int page) {
                    const uint32_t slot = n % kSlots;
                    // (all that can be done ahead of the wait is: a free slot is to be filled at once)
                    const int key = t * 128 + (lane >> 1) * p.box, row = key - paged_page(a, key) * a.page_size;
                    if (page < 0 || page >= a.n_pages) {
                        if (lane < boxes && key < w.u.len) record_status(a.status, RA_ERR_DEVICE_BOUNDS);
                        page = (int)a.n_pages;
                    }
                    const int c1 = p.rows_inner ? row : w.u.h, c2 = p.rows_inner ? w.u.h : row;
                    uint8_t *dst = base + kOffKV + slot * kTile + (lane & 1) * kHalf + (lane >> 1) * p.box * 128;
                    ok = mbar_wait_warp(kv_empty + slot, ((n / kSlots) & 1u) ^ 1u, wc);
                    if (!ok) return;
                    if (lane == 0) mbar_arrive_expect_tx(kv_full + slot, kTile);
                    __syncwarp();
                    if (lane < boxes) tma_load_4d_hint(dst, m, kv_full + slot, (lane & 1) * 64, c1, c2, page, policy);
                    ++n;
                };
                const int by = w.pair ? 1 : 2;
                // (the next step's pages are looked up ahead of this step's waits)
#pragma unroll 1
                for (int t = w.u.t0; t < w.tend && ok; t += by) {
                    const int cnt = !w.pair && t + 1 < w.tend ? 2 : 1;
                    const int pa0 = pa, pb0 = pb;
                    pa = w.pair ? pb : look_up(t + 2);
                    pb = look_up(t + by + 1);
#pragma unroll 1
                    for (int i = 0; i < 2 * cnt && ok; ++i) {
                        const bool v = i >= cnt;
                        const int j = v ? i - cnt : i;
                        load(v ? &p.tmV : &p.tmK, t + j, j ? pb0 : pa0);
                    }
                }
            }
            if (lane == 0) {
                // the last copies must have landed before the CTA may exit
                volatile int local_abort = 0;
                const WaitCtl drain{&local_abort, a.status, p.budget_ns};
                if (nq > 0) (void)mbar_wait(q_full, (nq - 1) & 1u, drain);
                for (uint32_t i = (n > kSlots ? n - kSlots : 0); i < n; ++i)
                    (void)mbar_wait(kv_full + (i % kSlots), (i / kSlots) & 1u, drain);
            }
        } else if (warp == 1) {
            // -------------------------------------------- MMA issuer
            const uint32_t idesc_s = idesc_bf16_f32(128, 128, 0, 0);
            const uint32_t idesc_o = idesc_bf16_f32(128, 128, 0, 1);
            // Q; the ring's first slot as K (rows of d) and as V (columns of d)
            const uint64_t dq = sdesc_sw128(base_s, 16, 1024), dk = sdesc_sw128(base_s + kOffKV, 16, 1024),
                           dv = sdesc_sw128(base_s + kOffKV, kHalf, 1024);
            uint32_t n = 0, np0 = 0, np1 = 0;  // tiles consumed; PVs issued per group (all units)
            int nu = 0;
            bool ok = true;
            auto full = [&](uint32_t i) {
                ok = ok && mbar_wait_warp(kv_full + i % kSlots, (i / kSlots) & 1u, wc);
                tc_fence_after();
                return (i % kSlots) * kTile;
            };
            auto empty = [&](uint32_t i) { tc_commit_w(kv_empty + i % kSlots); };
            for (Walk w; ok && next_unit(w);) {
                ok = mbar_wait_warp(q_full, nu & 1u, wc);
                ++nu;
                tc_fence_after();
                const int by = w.pair ? 1 : 2;
                // V rows behind the length, up to the end of their page, may hold anything
                auto clean = [&](int t, uint32_t i) {
                    const int live = w.u.len - t * 128;
                    if (live >= 128 || w.u.len == paged_page(a, w.u.len) * a.page_size) return;
                    uint8_t *v = base + kOffKV + (i % kSlots) * kTile;
                    for (int c = live * 8 + lane; c < 1024; c += 32) {
                        *reinterpret_cast<uint4 *>(v + c * 16) = make_uint4(0, 0, 0, 0);
                        *reinterpret_cast<uint4 *>(v + kHalf + c * 16) = make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                };
                if (w.u.t0 >= w.tend || !ok) {
                    tc_commit_w(q_empty);
                    continue;
                }
                // Step t: P V of the tiles t (group 0) and t + 1 (group 1; of t too where both have the same keys), and
                // S of the next step's, group by group.  The first step has no products, only its next step's S, so
                // that there is no second copy of that code: a run may be a dozen steps, and code that is met for the
                // first time costs more than it does (with a copy for the first S, the second one came 3500 ns after
                // it, now 2000).  Rolled over the groups too, that start is faster still, but every step slower: a
                // prefix of 65536 keys for 128 requests 256 us, 249 so.
#pragma unroll 1
                for (int t = w.u.t0 - by; t < w.tend && ok; t += by) {
                    const bool head = t < w.u.t0;
                    // the step's K tiles, then its V tiles, in the order of their loads
                    const uint32_t cnt = head ? 0u : !w.pair && t + 1 < w.tend ? 2u : 1u, next = n + 2 * cnt;
                    if (t + by >= w.tend) tc_commit_w(q_empty);  // every S of this unit is issued
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        if (!ok) break;
                        const int off = w.pair ? 0 : k;
                        const uint32_t tSk = tmem + 128u * k;
                        const bool last = k == 1 || !w.pair;  // reader of the tile
                        if (!head && t + off < w.tend) {
                            const uint32_t vi = n + cnt + off, v = full(vi);
                            if (!ok) break;
                            if (k == off) clean(t + off, vi);
                            ok = mbar_wait_warp(p_ready + k, (k ? np1 : np0) & 1u, wc);
                            if (!ok) break;
                            tc_fence_after();
                            issue_pv(tmem + 256u + 128u * k, tSk, desc_at(dv, v), idesc_o, t > w.u.t0);
                            if (t + by + off >= w.tend) tc_commit_w(o_done + k);  // the group's last of the unit
                            if (k)
                                ++np1;
                            else
                                ++np0;
                            if (last) empty(vi);
                        }
                        if (t + by + off < w.tend) {
                            const uint32_t ki = next + off, kt = full(ki);
                            if (!ok) break;
                            issue_s(tSk, desc_at(dq, w.pair && k ? kTile : 0u), desc_at(dk, kt), idesc_s);
                            tc_commit_w(s_full + k);
                            if (last) empty(ki);
                        }
                    }
                    n = next;
                }
            }
            // every MMA issued must have completed before TMEM is released
            tc_commit_w(mma_done);
            volatile int local_abort = 0;
            const WaitCtl drain{&local_abort, a.status, p.budget_ns};
            (void)mbar_wait_warp(mma_done, 0, drain);
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 200;\n" ::: "memory");
        // ------------------------------------------------ softmax / epilogue
        const int k = warp >= 8 ? 1 : 0;
        const int m = threadIdx.x - 128 - 128 * k;  // TMEM lane
        const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + lane_base + 128u * k;
        const uint32_t tO = tmem + lane_base + 256u + 128u * k;
        uint32_t nd_all = 0;  // S tiles of this group (all units)
        bool ok = true;
        float m_run = -INFINITY, l_run = 0.f;
        uint32_t nd = 0, no = 0;  // S tiles of this group in the unit; units with any
        // One tile: `seen` of its columns count for this row.  `live` is false
        // in the pass below that only warms the instruction cache.
        auto tile = [&](int seen, bool live) {
            const bool cut = __any_sync(0xffffffffu, seen < 128);
            float mx = -INFINITY;
            uint32_t v[kCols];
#pragma unroll 1
            for (int ch = kChunks - 1; ch >= 0; --ch) {  // (the first columns last: they stay for the exponentials)
                tmem_ld64(tS + kCols * ch, v);
                if (cut) mask_cols(v, seen, kCols * ch);
                float m4[4] = {mx, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int i = 0; i < kCols; i += 8) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        m4[j] = max3f(m4[j], __uint_as_float(v[i + j]), __uint_as_float(v[i + 4 + j]));
                }
                mx = max3f(fmaxf(m4[0], m4[1]), m4[2], m4[3]);
            }
            // the reference maximum moves only when it grew by more than 2^8: the final
            // scaling uses the same one, so the result is exact
            const float m_new = fmaxf(m_run, mx * a.scale_log2);
            const bool need = m_new > m_run + 8.0f;
            float alpha = 1.f;
            if (need) {
                alpha = ex2_approx(m_run - m_new);
                m_run = m_new;
                l_run *= alpha;
            }
            const float use = (m_run == -INFINITY) ? 0.f : m_run;
            const float2 sl2 = make_float2(a.scale_log2, a.scale_log2), nm2 = make_float2(-use, -use);
            float2 sum2 = make_float2(0.f, 0.f);
            // P replaces S column pair by column pair: P's columns of a chunk lie where S has been read.  It is rounded
            // to bf16 once, as in the packed ring (the sums use the unrounded values): results are off by 0.0023 of
            // their size, of which their own rounding is 0.0017.  What the rounding leaves of P as a second product
            // (in the columns that P leaves free) takes that away, but the products bound this kernel: a prefix of
            // 65536 keys for 128 requests 247 -> 330 us, 32768 for 64 73.7 -> 82.9.
#pragma unroll 1
            for (int ch = 0; ch < kChunks; ++ch) {
                uint32_t pk[kCols / 2];
                if (ch) {
                    tmem_ld64(tS + kCols * ch, v);
                    if (cut) mask_cols(v, seen, kCols * ch);
                }
                float2 sum4[2] = {sum2, make_float2(0.f, 0.f)};
#pragma unroll
                for (int c = 0; c < kCols / 2; ++c) {
                    const float2 e = fma2(make_float2(__uint_as_float(v[2 * c]), __uint_as_float(v[2 * c + 1])), sl2, nm2);
                    const float2 e2 = make_float2(ex2_approx(e.x), ex2_approx(e.y));
                    sum4[c & 1] = add2(sum4[c & 1], e2);
                    pk[c] = pack_bf16x2(e2.x, e2.y);
                }
                sum2 = add2(sum4[0], sum4[1]);
                if (live) tmem_st32(tS + kCols / 2 * ch, pk);
            }
            l_run += sum2.x + sum2.y;
            if (live) {
                // O is rescaled here: its last product finished before this S was computed
                if (nd > 0 && __any_sync(0xffffffffu, need)) {
#pragma unroll 1
                    for (int ch = 0; ch < 4; ++ch) {
                        uint32_t o[32];
                        tmem_ld32(tO + 32u * ch, o);
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                        tmem_st32(tO + 32u * ch, o);
                    }
                }
            }
        };
        // The first pass through this code fetches it from L2, which takes
        // longer than the pass itself.  So one pass runs on whatever TMEM holds
        // while the run is planned and the first keys are under way, without
        // storing anything (rolled halves and this together: a prefix of 32768
        // keys for 64 requests 90 -> 81 us).
#pragma unroll 1
        for (int dry = p.budget_ns != 0; ok; dry = 0) {  // (always so: a value that the compiler does not unroll by)
            Walk w;
            if (dry) {
                w.u.t0 = 0;
                w.tend = 1;
                w.pair = true;
                w.u.rows = 0;
            } else {
                if (!next_unit(w)) break;
            }
            const int by = w.pair ? 1 : 2;
            const int row = (w.pair ? 128 * k : 0) + m;  // of the unit
            const bool valid = row < w.u.rows;
            // (padding rows hold other tokens' queries or zeros: computed without masks, dropped)
            const int lim = dry ? 128 : valid ? paged_limit(a, w.u, p.fi, w.u.r0 + row) : w.u.len;
            // a warp of padding rows only keeps the barriers going
            const bool busy = dry || __any_sync(0xffffffffu, valid);
            m_run = -INFINITY;
            l_run = 0.f;
            nd = 0;
#pragma unroll 1
            for (int t = w.u.t0 + (w.pair ? 0 : k); t < w.tend; t += by) {
                if (!dry) {
                    ok = mbar_wait_warp(s_full + k, nd_all & 1u, wc);
                    if (!ok) break;
                    tc_fence_after();
                }
                if (busy) tile(lim - t * 128, !dry);
                if (dry) break;
                tc_fence_before();
                mbar_arrive(p_ready + k);
                ++nd;
                ++nd_all;
            }
            if (dry) {
                asm volatile("bar.sync 2, 384;" ::: "memory");  // the CTA's run is planned
                continue;
            }
            if (ok && nd > 0) {
                ok = mbar_wait_warp(o_done + k, no++ & 1u, wc);
                tc_fence_after();
            }
            // the partial: rows of group 1 lie behind group 0's when both have the same rows
            if (ok && busy) {
                const int64_t at = w.u.base + (int64_t)blockIdx.x * f.rt + (w.pair ? row : row + k * w.u.rows);
#pragma unroll 1
                for (int ch = 0; ch < 4 && nd > 0; ++ch) {
                    uint32_t v[32];
                    tmem_ld32(tO + 32u * ch, v);
                    if (valid) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            uint32_t o8[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) o8[e] = v[8 * i + e];
                            st_global_v8(f.acc + at * 128 + 32 * ch + 8 * i, o8);
                        }
                    }
                }
                if (valid) *reinterpret_cast<float2 *>(f.ml + at * 2) = make_float2(m_run, l_run);
            }
            // (O is next written by a later unit's first PV, which waits for this
            // thread's next P: the readout above comes first in program order)
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 2) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
    if (p.late) pdl_wait();
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    });
    return fn;
}

bool encode(CUtensorMap *m, const void *ptr, int rank, const cuuint64_t *dims, const cuuint64_t *strides,
            const cuuint32_t *box) {
    auto fn = encode_fn();
    if (!fn) return false;
    const cuuint32_t es[4] = {1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank, const_cast<void *>(ptr), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

// Boxes of whole 8-row swizzle groups that tile 128 keys or a page; rows of
// G heads that tile 128 rows; the maximum is taken before the scaling, so a
// positive scale; and a cache that a tensor map can describe.
bool paged_tc_maps(const PagedArgs &a, PagedMaps &m) {
    const int G = a.G, page = a.page_size;
    if (a.dtype != RA_BF16 || a.d != 128 || G > 128 || (G & (G - 1)) || !(a.scale_log2 > 0.f) || a.n_pages < 1 ||
        !(page >= 128 ? page % 128 == 0 : page >= 8 && 128 % page == 0))
        return false;
    const cuuint64_t qd[3] = {128, (cuuint64_t)a.Hq, (cuuint64_t)a.T};
    const cuuint64_t qs[2] = {256, (cuuint64_t)a.q_stride * 2};
    const cuuint32_t qb[3] = {64, (cuuint32_t)G, (cuuint32_t)(128 / G)};
    if (!encode(&m.q, a.q, 3, qd, qs, qb)) return false;
    m.rows_inner = a.head_stride > a.token_stride;
    const cuuint32_t box = (cuuint32_t)std::min(page, 128);
    cuuint64_t st[3] = {(cuuint64_t)a.head_stride * 2, (cuuint64_t)a.token_stride * 2, (cuuint64_t)a.page_stride * 2};
    cuuint64_t kd[4] = {128, (cuuint64_t)a.Hkv, (cuuint64_t)page, (cuuint64_t)a.n_pages};
    cuuint32_t kb[4] = {64, 1, box, 1};
    if (m.rows_inner) {
        std::swap(st[0], st[1]);
        std::swap(kd[1], kd[2]);
        std::swap(kb[1], kb[2]);
    }
    cuuint64_t least = 256;  // a one-element dimension has no stride: any that fits the others does
    for (int i = 0; i < 3; ++i) {
        if (kd[i + 1] == 1) st[i] = least;
        if (st[i] < least) return false;  // overlapping rows, or pages inside each other
        least = st[i] * kd[i + 1];
    }
    return encode(&m.k, a.k, 4, kd, st, kb) && encode(&m.v, a.v, 4, kd, st, kb);
}

cudaError_t launch_paged_tc(const PagedArgs &a, int fi, int late, const PagedMaps &m, cudaStream_t st) {
    TcParams p;
    memset(&p, 0, sizeof(p));
    p.tmQ = m.q;
    p.tmK = m.k;
    p.tmV = m.v;
    p.rows_inner = m.rows_inner;
    p.a = a;
    p.fi = fi;
    p.late = late;
    p.box = std::min(a.page_size, 128);
    while ((1 << p.log2G) < a.G) ++p.log2G;
    p.budget_ns = wait_budget_ns();
    static std::atomic<bool> attr_set[128] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 128 || !attr_set[dev]) {
        e = cudaFuncSetAttribute((const void *)paged_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e != cudaSuccess) return e;
        // The register split draws on the 384 x 168 of the launch: with fewer, the increase could never be granted.
        cudaFuncAttributes fa;
        e = cudaFuncGetAttributes(&fa, (const void *)paged_tc_kernel);
        if (e != cudaSuccess) return e;
        if (fa.numRegs < 168) return cudaErrorInvalidConfiguration;
        if (dev >= 0 && dev < 128) attr_set[dev] = true;
    }
    return launch_pdl(paged_tc_kernel, a.f[fi].n, kThreads, kSmem, st, p);
}

}  // namespace ra

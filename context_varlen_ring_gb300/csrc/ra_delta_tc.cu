// ra_delta_tc.cu -- the gated delta rule's walk along a sequence's chunks on
// the 5th-generation tensor cores (bf16, heads of 128): the formulas are in
// ra_delta.cu, T and P come from its first kernel.
//
// Bound: the chain of a sequence.  A chunk's products (K S0, T R, K^T u, and for
// the output Q S0 and P u) follow one another, and the next chunk needs their
// result; a batch's longest sequence is a chain of hundreds of them (24 sequences
// of 32768 tokens, 16 heads, the longest 7422: 547 us, 9000 cycles a chunk, of
// which the products take a third and what they wait for the rest).  So a CTA
// has one head of one sequence, with the whole state, and everything is held
// the other way round (a column of v to a TMEM lane): the state is the A operand
// of the first product straight from TMEM, its tokens' values the A operand of
// the next, K, Q, T and P the B operands from shared memory as they come by TMA
// and bulk copies, and no result is transposed or passes through shared memory.
//  * warp 0 loads, warp 1 issues products, warp 3 makes the gates; two
//    warpgroups, a thread a lane and half of the columns each, hold the state
//    in registers (fp32), make bf16 parts of what the next product reads and
//    put them into TMEM.
//  * the output's last product runs behind those that the chain needs; its
//    operand lies in the state's columns, so the output is read ahead of the
//    next chunk's state.
// TMEM columns: 0 the state's growth (and, ahead of it, R's parts); 128 K S0,
// then u; 192 Q S0; 256 the state's parts, then those of e^(G_63 - G) u and of u;
// 448 P u.
// Every wait is bounded as in the rest of the library.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <atomic>
#include <cstring>
#include <mutex>

#include "ra_delta.cuh"
#include "ra_delta_maps.h"
#include "ra_internal.h"
#include "ra_serve.cuh"

namespace ra {
namespace {

using namespace delta;

constexpr int kThreads = 384;
constexpr int kD = 128;                   // dk = dv
constexpr int kStages = 2;
constexpr uint32_t kHalf = 16384;         // 64 rows of K, 64 of Q, 128 bytes each (half of dk)
constexpr uint32_t kSquare = 8192;        // a part of T or P
constexpr uint32_t kValues = C * kD * 2;  // [64][128] of v

constexpr uint32_t kOffTP = 2 * kHalf, kOffV = kOffTP + 2 * NP * kSquare, kStage = kOffV + kValues;
constexpr uint32_t kOffBar = kStages * kStage, kSmem = kOffBar + 256 + 1024;
constexpr int kColD = 0, kColX = 128, kColQ = 192, kColS = 256, kColP = 448;
// u's parts, behind e^(G_63 - G) u's over the state's, which are written again only when the output's products are done.
constexpr int kColU = kColS + 32 * NP;

struct ScanParams {
    CUtensorMap tmQ, tmK, tmV, tmO;  // tmO: dout
    DeltaArgs a;
    unsigned long long budget_ns;
};

// registers -> TMEM: 32 lanes x 16 columns; complete behind tmem_put_wait.
__device__ __forceinline__ void tmem_put16(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]),
        "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}
__device__ __forceinline__ void tmem_put_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// 2 N floats into bf16 pairs, and what that leaves of them.
template <int N>
__device__ __forceinline__ void part(float2 (&x)[N], uint32_t (&h)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        h[i] = pack_bf16x2(x[i].x, x[i].y);
        x[i] = fma2(make_float2(__uint_as_float(h[i] << 16), __uint_as_float(h[i] & 0xffff0000u)), make_float2(-1.f, -1.f), x[i]);
    }
}
// 32 values as NP parts of 16 columns, `apart` columns from each other (to be waited for).
__device__ __forceinline__ void put_parts(uint32_t tmem, int apart, float2 (&x)[16]) {
#pragma unroll
    for (int p = 0; p < NP; ++p) {
        uint32_t h[16];
        if (p + 1 < NP) {
            part<16>(x, h);
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) h[i] = pack_bf16x2(x[i].x, x[i].y);
        }
        tmem_put16(tmem + p * apart, h);
    }
}
__device__ __forceinline__ float2 f2(uint32_t x, uint32_t y) { return make_float2(__uint_as_float(x), __uint_as_float(y)); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return fma2(a, b, make_float2(0.f, 0.f)); }

// The products, issued by unrolled code (rolled, an issue takes longer than a product of 64 columns: 32768 tokens of two
// parts 390 -> 527 us; rolled over the parts alone, the backward's walks 330 -> 346), all of one by one thread (chosen
// anew for each instruction, with two parts 350 us; so 304).
// D [v, token] = A's NP parts [v, dk] (64 columns a part) by 64 rows of K or Q (descriptor b).
__device__ __forceinline__ void mma_state(uint32_t d, uint32_t x, uint64_t b, uint32_t idesc) {
    if (elected()) {
        bool more = false;
#pragma unroll
        for (int q = NP - 1; q >= 0; --q)
#pragma unroll
            for (int ks = 0; ks < 8; ++ks) {
                tc_mma_ts(d, x + 64 * q + 8 * ks, b + (((uint32_t)(ks >> 2) * kHalf + (uint32_t)(ks & 3) * 32u) >> 4), idesc, more);
                more = true;
            }
    }
    __syncwarp();
}
// D [v, token] = A's NP parts [v, token] (32 columns a part) by T's or P's parts, `step` bytes apart from 16 tokens to
// the next; products of parts i, j with i + j < NP, the small ones first.
__device__ __forceinline__ void mma_square(uint32_t d, uint32_t x, uint64_t b, uint32_t step, uint32_t idesc) {
    if (elected()) {
        bool more = false;
#pragma unroll
        for (int o = NP - 1; o >= 0; --o)
#pragma unroll
            for (int q = 0; q <= o; ++q)
#pragma unroll
                for (int ks = 0; ks < 4; ++ks) {
                    tc_mma_ts(d, x + 32 * q + 8 * ks, b + (((uint32_t)(o - q) * kSquare + (uint32_t)ks * step) >> 4), idesc, more);
                    more = true;
                }
    }
    __syncwarp();
}
// D [v, dk] (+)= A's NP parts [v, token] by 64 rows of K or Q, their dk as columns.
__device__ __forceinline__ void mma_rows(uint32_t d, uint32_t x, uint64_t b, uint32_t idesc, bool more) {
    if (elected()) {
#pragma unroll
        for (int q = NP - 1; q >= 0; --q)
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) {
                tc_mma_ts(d, x + 32 * q + 8 * ks, b + ((uint32_t)ks * 2048u >> 4), idesc, more);
                more = true;
            }
    }
    __syncwarp();
}

// With the output (a forward), or keeping what the gradients need of each chunk (decided here, not in the loop: with two
// parts 365 -> 352 us; what is kept is stored behind the arrivals that the chain waits for).
template <bool KEEP>
__device__ __forceinline__ void scan_body(const ScanParams &p, const int block) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ Gates gates[2];
    const DeltaArgs &a = p.a;
    const uint32_t raw_s = smem_u32(smem_raw), base_s = (raw_s + 1023u) & ~1023u;
    uint8_t *base = smem_raw + (base_s - raw_s);
    uint64_t *bars = reinterpret_cast<uint64_t *>(base + kOffBar);
    uint64_t *full = bars + 0;      // [2] a chunk's rows landed
    uint64_t *empty = bars + 2;     // [2] its products are done, its values read
    uint64_t *g_full = bars + 4;    // [2] its gates
    uint64_t *g_empty = bars + 6;   // [2]
    uint64_t *s_ready = bars + 8;   // the state's parts are in TMEM
    uint64_t *x_full = bars + 9;    // K S0 is there
    uint64_t *r_ready = bars + 10;  // R's parts
    uint64_t *u_full = bars + 11;   // u is there
    uint64_t *u_ready = bars + 12;  // u's parts
    uint64_t *d_full = bars + 13;   // the state's growth is there
    uint64_t *o_full = bars + 14;   // the output is there
    uint64_t *o_empty = bars + 15;  // and read
    uint64_t *mma_done = bars + 16;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 17);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(bars + 18);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        *abort_flag = 0;
        for (int i = 0; i < kStages; ++i) {
            mbar_init(full + i, 1);
            mbar_init(empty + i, 1 + 8);
            mbar_init(g_full + i, 1);
            mbar_init(g_empty + i, 8);
        }
        mbar_init(s_ready, 256);
        mbar_init(x_full, 1);
        mbar_init(r_ready, 256);
        mbar_init(u_full, 1);
        mbar_init(u_ready, 256);
        mbar_init(d_full, 1);
        mbar_init(o_full, 1);
        mbar_init(o_empty, 256);
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
    wait_ahead();
    constexpr bool keep = KEEP, want = !KEEP;
    const bool bad = a.hdr->bad != 0;  // (boundaries without a plan: nothing is written)
    const int seq = bad ? 0 : a.order[block / a.Hv], h = block % a.Hv, hk = h / (a.Hv / a.Hk);
    const int c0 = bad ? 0 : a.first[seq], n_chunks = bad ? 0 : a.first[seq + 1] - c0;
    const uint32_t tmem = *tmem_slot;
    const WaitCtl wc{abort_flag, a.status, p.budget_ns};

    // Registers: 128 x 80 + 256 x 200 = 61440, within the 384 x 168 = 64512 of the launch.
    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 80;\n" ::: "memory");
        if (warp == 0) {
            // -------------------------------------------- loads
            if (lane == 0) {
                int i = 0;
                for (bool ok = true; i < n_chunks; ++i) {
                    const int s = i & 1;
                    const int64_t c = c0 + i;
                    const int tok = a.chunk[c].tok0;
                    uint8_t *st = base + s * kStage;
                    ok = mbar_wait(empty + s, ((i >> 1) & 1u) ^ 1u, wc);
                    if (!ok) break;
                    const uint32_t squares = (want ? 2 : 1) * NP * kSquare;
                    mbar_arrive_expect_tx(full + s, (want ? 4 : 2) * (kHalf / 2) + squares + kValues);
                    for (int d = 0; d < 2; ++d) tma_load_3d(st + d * kHalf, &p.tmK, full + s, d * 64, hk, tok);
                    tma_load_3d(st + kOffV, &p.tmV, full + s, 0, h, tok);
                    bulk_load(st + kOffTP, a.tp + (c * a.Hv + h) * 2 * NP * C * C, squares, full + s);
                    if (want)
                        for (int d = 0; d < 2; ++d)
                            tma_load_3d(st + d * kHalf + kHalf / 2, &p.tmQ, full + s, d * 64, hk, tok);
                }
                // the last copies must have landed before the CTA may exit
                volatile int local_abort = 0;
                const WaitCtl drain{&local_abort, a.status, p.budget_ns};
                for (int j = i > 2 ? i - 2 : 0; j < i; ++j) (void)mbar_wait(full + (j & 1), (j >> 1) & 1u, drain);
            }
        } else if (warp == 1) {
            // -------------------------------------------- products
            const uint32_t id64 = idesc_bf16_f32(128, 64, 0, 0), id128k = idesc_bf16_f32(128, 128, 0, 0), id128 = idesc_bf16_f32(128, 128, 0, 1);
            bool ok = true;
            for (int i = 0; i < n_chunks && ok; ++i) {
                const int s = i & 1;
                const uint32_t st = base_s + s * kStage, ph = i & 1u;
                const uint64_t dK = sdesc_sw128(st, 16, 1024);
                const uint64_t dKn = sdesc_sw128(st, kHalf, 1024);  // columns of dk
                const uint64_t dT = sdesc_sw128(st + kOffTP, 16, 1024), dP = sdesc_sw128(st + kOffTP + NP * kSquare, 16, 1024);
                ok = mbar_wait_warp(full + s, (i >> 1) & 1u, wc);
                if (!ok) break;
                const int n = a.chunk[c0 + i].n;
                if (n < C) {  // rows of K behind the sequence's end are another's, or none
                    uint8_t *k = base + s * kStage;
                    for (int x = n * 8 + lane; x < C * 8; x += 32) {
                        *reinterpret_cast<uint4 *>(k + x * 16) = make_uint4(0, 0, 0, 0);
                        *reinterpret_cast<uint4 *>(k + kHalf + x * 16) = make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                ok = mbar_wait_warp(s_ready, ph, wc);
                if (!ok) break;
                tc_fence_after();
                if (want && i > 0) {  // (the last output is read)
                    ok = mbar_wait_warp(o_empty, (i - 1) & 1u, wc);
                    if (!ok) break;
                    tc_fence_after();
                }
                mma_state(tmem + kColX, tmem + kColS, dK, want ? id128k : id64);  // K S0, and Q S0 with it
                tc_commit_w(x_full);
                ok = mbar_wait_warp(r_ready, ph, wc);
                if (!ok) break;
                tc_fence_after();
                mma_square(tmem + kColX, tmem + kColD, dT, 32, id64);
                tc_commit_w(u_full);
                ok = mbar_wait_warp(u_ready, ph, wc);
                if (!ok) break;
                tc_fence_after();
                mma_rows(tmem + kColD, tmem + kColS, dKn, id128, false);
                tc_commit_w(d_full);
                if (want) {
                    mma_square(tmem + kColP, tmem + kColU, dP, 32, id64);
                    tc_commit_w(o_full);
                }
                tc_commit_w(empty + s);
            }
            // every product issued must have completed before TMEM is released
            tc_commit_w(mma_done);
            volatile int local_abort = 0;
            const WaitCtl drain{&local_abort, a.status, p.budget_ns};
            (void)mbar_wait_warp(mma_done, 0, drain);
        } else if (warp == 3) {
            // -------------------------------------------- gates
            float g[2], b[2];
            if (n_chunks > 0) gates_load(a, a.chunk[c0], h, g, b);
            for (int i = 0; i < n_chunks; ++i) {
                if (!mbar_wait_warp(g_empty + (i & 1), ((i >> 1) & 1u) ^ 1u, wc)) break;
                gates_put(gates[i & 1], g, b);
                __syncwarp();
                if (lane == 0) mbar_arrive(g_full + (i & 1));
                if (i + 1 < n_chunks) gates_load(a, a.chunk[c0 + i + 1], h, g, b);
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 200;\n" ::: "memory");
        // ------------------------------------------------ the state, and what the products read
        const int half = warp >= 8 ? 1 : 0, m = (warp & 3) * 32 + lane;  // TMEM lane: the column of v
        const uint32_t at = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const int64_t slot = !bad && (a.state || a.state_out) ? slot_of(a.slots, a.n_slots, seq, a.status) : -1;
        const int64_t place = ((slot * a.Hv + h) * kD + 64 * half) * kD + m;
        float2 S[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            const bool there = a.state && slot >= 0;
            S[j] = make_float2(there ? a.state[place + 2 * j * kD] : 0.f, there ? a.state[place + (2 * j + 1) * kD] : 0.f);
        }
        bool ok = true;
        // four of the gates of this thread's tokens
        auto four = [&](const float (&x)[C], int j) { return *reinterpret_cast<const float4 *>(x + 32 * half + 4 * j); };
        // the output of chunk i, scale e^G (Q S0) + P u: 16 of this thread's 32 tokens
        auto output = [&](int i, const DeltaChunk &ch, int e) {
            if (e == 0) {
                ok = mbar_wait_warp(o_full, i & 1u, wc);
                if (!ok) return;
                tc_fence_after();
            }
            uint32_t x[16], y[16];
            tmem_ld16x2(at + kColQ + 32 * half + 16 * e, at + kColP + 32 * half + 16 * e, x, y);
            if (e) {
                tc_fence_before();
                mbar_arrive(o_empty);
            }
            const Gates &g = gates[i & 1];
            const int64_t stride = (int64_t)a.Hv * kD;
            const int first = 32 * half + 16 * e, rows = ch.n - first;
            bf16 *o = static_cast<bf16 *>(a.out) + ((int64_t)(ch.tok0 + first) * a.Hv + h) * kD + m;
            auto put = [&](bool all) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float4 d = four(g.eG, 4 * e + j);
                    const float2 s = make_float2(a.scale, a.scale);
                    const float2 p0 = fma2(mul2(s, make_float2(d.x, d.y)), f2(x[4 * j], x[4 * j + 1]), f2(y[4 * j], y[4 * j + 1]));
                    const float2 p1 = fma2(mul2(s, make_float2(d.z, d.w)), f2(x[4 * j + 2], x[4 * j + 3]), f2(y[4 * j + 2], y[4 * j + 3]));
                    if (all || 4 * j < rows) o[0] = __float2bfloat16_rn(p0.x);
                    if (all || 4 * j + 1 < rows) o[stride] = __float2bfloat16_rn(p0.y);
                    if (all || 4 * j + 2 < rows) o[2 * stride] = __float2bfloat16_rn(p1.x);
                    if (all || 4 * j + 3 < rows) o[3 * stride] = __float2bfloat16_rn(p1.y);
                    o += 4 * stride;
                }
            };
            if (rows >= 16)
                put(true);
            else
                put(false);
            if (e) {
                __syncwarp();
                if (lane == 0) mbar_arrive(g_empty + (i & 1));
            }
        };
        // chunk i's values, pairs of tokens as they are: taken while the chunk ahead waits for its products
        uint32_t d[16];
        auto take = [&](int i) {
            ok = mbar_wait_warp(full + (i & 1), (i >> 1) & 1u, wc);
            if (!ok) return;
            const uint16_t *x = reinterpret_cast<const uint16_t *>(base + (i & 1) * kStage + kOffV) + 32 * half * kD + m;
#pragma unroll
            for (int j = 0; j < 16; ++j) d[j] = x[2 * j * kD] | (uint32_t)x[(2 * j + 1) * kD] << 16;
            const int rows = a.chunk[c0 + i].n - 32 * half;
            if (rows < 32) {  // (rows behind the sequence's end are another's, or none)
#pragma unroll
                for (int j = 0; j < 16; ++j) d[j] = 2 * j + 1 < rows ? d[j] : 2 * j < rows ? d[j] & 0xffffu : 0u;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(empty + (i & 1));
        };
        if (n_chunks > 0) take(0);
        DeltaChunk ch{0, 0}, last;
#pragma unroll 1
        for (int i = 0; i < n_chunks && ok; ++i) {
            const int s = i & 1;
            const uint32_t ph = i & 1u;
            const int64_t cell = (int64_t)(c0 + i) * a.Hv + h;
            last = ch;
            ch = a.chunk[c0 + i];
            if (want && i > 0) {
                output(i - 1, last, 0);
                if (!ok) break;
                output(i - 1, last, 1);
            }
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                float2 x[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) x[j] = S[16 * q + j];
                put_parts(at + kColS + 32 * half + 16 * q, 64, x);
            }
            tmem_put_wait();
            tc_fence_before();
            mbar_arrive(s_ready);
            if (keep) {
                float *p = a.s0 + (cell * kD + 64 * half) * kD + m;
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    p[2 * j * kD] = S[j].x;
                    p[(2 * j + 1) * kD] = S[j].y;
                }
            }
            ok = mbar_wait_warp(g_full + s, (i >> 1) & 1u, wc);
            if (!ok) break;
            const Gates &g = gates[s];
            ok = mbar_wait_warp(x_full, ph, wc);
            if (!ok) break;
            tc_fence_after();
            float2 v[16], r[16];
            {
                uint32_t x[32];
                tmem_ld32(at + kColX + 32 * half, x);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float4 e = four(g.eG, j), b = four(g.beta, j);
                    const float2 r0 = fma2(make_float2(-e.x, -e.y), f2(x[4 * j], x[4 * j + 1]), f2(d[2 * j] << 16, d[2 * j] & 0xffff0000u));
                    const float2 r1 = fma2(make_float2(-e.z, -e.w), f2(x[4 * j + 2], x[4 * j + 3]), f2(d[2 * j + 1] << 16, d[2 * j + 1] & 0xffff0000u));
                    if (keep) {
                        r[2 * j] = r0;
                        r[2 * j + 1] = r1;
                    }
                    v[2 * j] = mul2(make_float2(b.x, b.y), r0);
                    v[2 * j + 1] = mul2(make_float2(b.z, b.w), r1);
                }
            }
            put_parts(at + kColD + 16 * half, 32, v);
            tmem_put_wait();
            tc_fence_before();
            mbar_arrive(r_ready);
            if (keep) {
                float *p = a.r + (cell * C + 32 * half) * kD + m;
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    p[2 * j * kD] = r[j].x;
                    p[(2 * j + 1) * kD] = r[j].y;
                }
            }
            ok = mbar_wait_warp(u_full, ph, wc);
            if (!ok) break;
            tc_fence_after();
            {
                uint32_t x[32];
                float2 y[16];
                tmem_ld32(at + kColX + 32 * half, x);
                float *p = a.u + (cell * C + 32 * half) * kD + m;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float4 e = four(g.eL, j);
                    v[2 * j] = f2(x[4 * j], x[4 * j + 1]);
                    v[2 * j + 1] = f2(x[4 * j + 2], x[4 * j + 3]);
                    y[2 * j] = mul2(make_float2(e.x, e.y), v[2 * j]);
                    y[2 * j + 1] = mul2(make_float2(e.z, e.w), v[2 * j + 1]);
                }
                put_parts(at + kColS + 16 * half, 32, y);
                if (want) put_parts(at + kColU + 16 * half, 32, v);
                tmem_put_wait();
                tc_fence_before();
                mbar_arrive(u_ready);
                if (keep) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        p[2 * j * kD] = v[j].x;
                        p[(2 * j + 1) * kD] = v[j].y;
                    }
                }
            }
            const float2 eC = make_float2(g.eC, g.eC);
            if (!want) {
                __syncwarp();
                if (lane == 0) mbar_arrive(g_empty + s);
            }
            if (i + 1 < n_chunks) {
                take(i + 1);
                if (!ok) break;
            }
            ok = mbar_wait_warp(d_full, ph, wc);
            if (!ok) break;
            tc_fence_after();
            {
                uint32_t x[64];
                tmem_ld64(at + kColD + 64 * half, x);
#pragma unroll
                for (int j = 0; j < 32; ++j) S[j] = fma2(eC, S[j], f2(x[2 * j], x[2 * j + 1]));
            }
        }
        if (ok && want && n_chunks > 0) {
            output(n_chunks - 1, ch, 0);
            if (ok) output(n_chunks - 1, ch, 1);
        }
        if (ok && !bad && a.state_out && slot >= 0) {
#pragma unroll
            for (int j = 0; j < 32; ++j) {
                a.state_out[place + 2 * j * kD] = S[j].x;
                a.state_out[place + (2 * j + 1) * kD] = S[j].y;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 2) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ------------------------------------------------------------ the walk from the end
// The gradient's walk (formulas in ra_delta_bwd.cu), held the same way: dS^T as A
// operand against K, its tokens' gradients against T and P with their rows as
// the products' depth, and then against K and Q.  What needs no state (P^T do,
// Q^T do) runs beside the conversions of the chain.
// TMEM columns: 0 the growth of dS; 128 K dS; 192 P^T do; 256 dS's parts, then
// du's and, behind them, scale e^G do's; in du's place -beta e^G dR's; 448 do.
__device__ __forceinline__ void back_body(const ScanParams &p, const int block) {
    constexpr int kColY = 192, kColZ = kColS, kColW = kColS + 32 * NP, kColDO = 448;
    static_assert(kColS + 64 * NP <= kColDO, "columns");
    extern __shared__ uint8_t smem_raw[];
    __shared__ Gates gates[2];
    const DeltaArgs &a = p.a;
    const uint32_t raw_s = smem_u32(smem_raw), base_s = (raw_s + 1023u) & ~1023u;
    uint8_t *base = smem_raw + (base_s - raw_s);
    uint64_t *bars = reinterpret_cast<uint64_t *>(base + kOffBar);
    uint64_t *full = bars + 0;      // [2] a chunk's rows landed
    uint64_t *empty = bars + 2;     // [2] its products are done, its do read
    uint64_t *g_full = bars + 4;    // [2] its gates
    uint64_t *g_empty = bars + 6;   // [2]
    uint64_t *y_ready = bars + 8;   // do is in TMEM
    uint64_t *s_ready = bars + 9;   // dS's parts
    uint64_t *x_full = bars + 10;   // K dS and P^T do are there
    uint64_t *r_ready = bars + 11;  // du's parts
    uint64_t *w_ready = bars + 18;  // scale e^G do's (apart from du's, which the chain waits for: 320 -> 307 us)
    uint64_t *u_full = bars + 12;   // dR is there
    uint64_t *z_ready = bars + 13;  // -beta e^G dR's parts
    uint64_t *d_full = bars + 14;   // the growth of dS is there
    uint64_t *mma_done = bars + 15;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 16);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(bars + 17);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        *abort_flag = 0;
        for (int i = 0; i < kStages; ++i) {
            mbar_init(full + i, 1);
            mbar_init(empty + i, 1 + 8);
            mbar_init(g_full + i, 1);
            mbar_init(g_empty + i, 8);
        }
        mbar_init(y_ready, 256);
        mbar_init(s_ready, 256);
        mbar_init(x_full, 1);
        mbar_init(r_ready, 256);
        mbar_init(w_ready, 256);
        mbar_init(u_full, 1);
        mbar_init(z_ready, 256);
        mbar_init(d_full, 1);
        mbar_init(mma_done, 1);
        fence_mbar_init();
        tma_prefetch_desc(&p.tmQ);
        tma_prefetch_desc(&p.tmK);
        tma_prefetch_desc(&p.tmO);
    }
    if (warp == 2) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    wait_ahead();
    const bool bad = a.hdr->bad != 0;
    const int seq = bad ? 0 : a.order[block / a.Hv], h = block % a.Hv, hk = h / (a.Hv / a.Hk);
    const int c0 = bad ? 0 : a.first[seq], n_chunks = bad ? 0 : a.first[seq + 1] - c0, c1 = c0 + n_chunks - 1;
    const uint32_t tmem = *tmem_slot;
    const WaitCtl wc{abort_flag, a.status, p.budget_ns};

    // Registers: 128 x 80 + 256 x 200 = 61440, within the 384 x 168 = 64512 of the launch.
    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 80;\n" ::: "memory");
        if (warp == 0) {
            // -------------------------------------------- loads
            if (lane == 0) {
                int i = 0;
                for (bool ok = true; i < n_chunks; ++i) {
                    const int s = i & 1;
                    const int64_t c = c1 - i;
                    const int tok = a.chunk[c].tok0;
                    uint8_t *st = base + s * kStage;
                    ok = mbar_wait(empty + s, ((i >> 1) & 1u) ^ 1u, wc);
                    if (!ok) break;
                    mbar_arrive_expect_tx(full + s, 2 * kHalf + 2 * NP * kSquare + kValues);
                    for (int d = 0; d < 2; ++d) {
                        tma_load_3d(st + d * kHalf, &p.tmK, full + s, d * 64, hk, tok);
                        tma_load_3d(st + d * kHalf + kHalf / 2, &p.tmQ, full + s, d * 64, hk, tok);
                    }
                    tma_load_3d(st + kOffV, &p.tmO, full + s, 0, h, tok);
                    bulk_load(st + kOffTP, a.tp + (c * a.Hv + h) * 2 * NP * C * C, 2 * NP * kSquare, full + s);
                }
                // the last copies must have landed before the CTA may exit
                volatile int local_abort = 0;
                const WaitCtl drain{&local_abort, a.status, p.budget_ns};
                for (int j = i > 2 ? i - 2 : 0; j < i; ++j) (void)mbar_wait(full + (j & 1), (j >> 1) & 1u, drain);
            }
        } else if (warp == 1) {
            // -------------------------------------------- products
            const uint32_t id64 = idesc_bf16_f32(128, 64, 0, 0), id64n = idesc_bf16_f32(128, 64, 0, 1),
                           id128n = idesc_bf16_f32(128, 128, 0, 1);
            bool ok = true;
            for (int i = 0; i < n_chunks && ok; ++i) {
                const int s = i & 1;
                const uint32_t st = base_s + s * kStage, ph = i & 1u;
                const uint64_t dK = sdesc_sw128(st, 16, 1024);
                const uint64_t dKn = sdesc_sw128(st, kHalf, 1024), dQn = sdesc_sw128(st + kHalf / 2, kHalf, 1024);  // columns of dk
                const uint64_t dT = sdesc_sw128(st + kOffTP, kHalf, 1024), dP = sdesc_sw128(st + kOffTP + NP * kSquare, kHalf, 1024);
                ok = mbar_wait_warp(full + s, (i >> 1) & 1u, wc);
                if (!ok) break;
                const int n = a.chunk[c1 - i].n;
                if (n < C) {  // rows of K and Q behind the sequence's end are another's, or none
                    uint8_t *k = base + s * kStage;
                    for (int x = n * 8 + lane; x < C * 8; x += 32)
#pragma unroll
                        for (int e = 0; e < 4; ++e) *reinterpret_cast<uint4 *>(k + e * (kHalf / 2) + x * 16) = make_uint4(0, 0, 0, 0);
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                ok = mbar_wait_warp(y_ready, ph, wc);
                if (!ok) break;
                tc_fence_after();
                if (elected()) {
#pragma unroll
                    for (int x = 0; x < 4 * NP; ++x) {  // do by P's rows, the small parts first
                        const uint32_t q = NP - 1 - x / 4, ks = x % 4;
                        tc_mma_ts(tmem + kColY, tmem + kColDO + 8 * ks, dP + ((q * kSquare + ks * 2048u) >> 4), id64n, x > 0);
                    }
                }
                __syncwarp();
                ok = mbar_wait_warp(s_ready, ph, wc);
                if (!ok) break;
                tc_fence_after();
                mma_state(tmem + kColX, tmem + kColS, dK, id64);
                tc_commit_w(x_full);
                ok = mbar_wait_warp(r_ready, ph, wc);
                if (!ok) break;
                tc_fence_after();
                mma_square(tmem + kColX, tmem + kColZ, dT, 2048, id64n);
                tc_commit_w(u_full);
                ok = mbar_wait_warp(w_ready, ph, wc);
                if (!ok) break;
                tc_fence_after();
                mma_rows(tmem + kColD, tmem + kColW, dQn, id128n, false);
                ok = mbar_wait_warp(z_ready, ph, wc);
                if (!ok) break;
                tc_fence_after();
                mma_rows(tmem + kColD, tmem + kColZ, dKn, id128n, true);
                tc_commit_w(d_full);
                tc_commit_w(empty + s);
            }
            // every product issued must have completed before TMEM is released
            tc_commit_w(mma_done);
            volatile int local_abort = 0;
            const WaitCtl drain{&local_abort, a.status, p.budget_ns};
            (void)mbar_wait_warp(mma_done, 0, drain);
        } else if (warp == 3) {
            // -------------------------------------------- gates
            float g[2], b[2];
            if (n_chunks > 0) gates_load(a, a.chunk[c1], h, g, b);
            for (int i = 0; i < n_chunks; ++i) {
                if (!mbar_wait_warp(g_empty + (i & 1), ((i >> 1) & 1u) ^ 1u, wc)) break;
                gates_put(gates[i & 1], g, b);
                __syncwarp();
                if (lane == 0) mbar_arrive(g_full + (i & 1));
                if (i + 1 < n_chunks) gates_load(a, a.chunk[c1 - i - 1], h, g, b);
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 200;\n" ::: "memory");
        // ------------------------------------------------ dS, and what the products read
        const int half = warp >= 8 ? 1 : 0, m = (warp & 3) * 32 + lane;  // TMEM lane: the column of v
        const uint32_t at = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const int64_t place = (((int64_t)seq * a.Hv + h) * kD + 64 * half) * kD + m;
        float2 S[32];
#pragma unroll
        for (int j = 0; j < 32; ++j)
            S[j] = make_float2(a.dstate ? a.dstate[place + 2 * j * kD] : 0.f, a.dstate ? a.dstate[place + (2 * j + 1) * kD] : 0.f);
        bool ok = true;
        auto four = [&](const float (&x)[C], int j) { return *reinterpret_cast<const float4 *>(x + 32 * half + 4 * j); };
        // chunk i's do: pairs of tokens, as they are (one part), into registers and TMEM
        uint32_t d[16];
        auto take = [&](int i) {
            ok = mbar_wait_warp(full + (i & 1), (i >> 1) & 1u, wc);
            if (!ok) return;
            const int rows = a.chunk[c1 - i].n - 32 * half;
            const uint16_t *x = reinterpret_cast<const uint16_t *>(base + (i & 1) * kStage + kOffV) + 32 * half * kD + m;
#pragma unroll
            for (int j = 0; j < 16; ++j)  // (rows behind the sequence's end are another's, or none)
                d[j] = (2 * j < rows ? x[2 * j * kD] : 0u) | (2 * j + 1 < rows ? (uint32_t)x[(2 * j + 1) * kD] << 16 : 0u);
            tmem_put16(at + kColDO + 16 * half, d);
            tmem_put_wait();
            tc_fence_before();
            mbar_arrive(y_ready);
            __syncwarp();
            if (lane == 0) mbar_arrive(empty + (i & 1));
        };
        if (n_chunks > 0) take(0);
#pragma unroll 1
        for (int i = 0; i < n_chunks && ok; ++i) {
            const int s = i & 1;
            const uint32_t ph = i & 1u;
            const int64_t cell = (int64_t)(c1 - i) * a.Hv + h;
            const DeltaChunk ch = a.chunk[c1 - i];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                float2 x[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) x[j] = S[16 * q + j];
                put_parts(at + kColS + 32 * half + 16 * q, 64, x);
            }
            tmem_put_wait();
            tc_fence_before();
            mbar_arrive(s_ready);
            {
                float *o = a.ds + (cell * kD + 64 * half) * kD + m;
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    o[2 * j * kD] = S[j].x;
                    o[(2 * j + 1) * kD] = S[j].y;
                }
            }
            ok = mbar_wait_warp(g_full + s, (i >> 1) & 1u, wc) && mbar_wait_warp(x_full, ph, wc);
            if (!ok) break;
            tc_fence_after();
            const Gates &g = gates[s];
            {
                uint32_t x[32], y[32];
                float2 v[16];
                tmem_ld32x2(at + kColX + 32 * half, at + kColY + 32 * half, x, y);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float4 e = four(g.eL, j);
                    v[2 * j] = fma2(make_float2(e.x, e.y), f2(x[4 * j], x[4 * j + 1]), f2(y[4 * j], y[4 * j + 1]));
                    v[2 * j + 1] = fma2(make_float2(e.z, e.w), f2(x[4 * j + 2], x[4 * j + 3]), f2(y[4 * j + 2], y[4 * j + 3]));
                }
                put_parts(at + kColZ + 16 * half, 32, v);
                tmem_put_wait();
                tc_fence_before();
                mbar_arrive(r_ready);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float4 e = four(g.eG, j);
                    v[2 * j] = mul2(make_float2(a.scale * e.x, a.scale * e.y), f2(d[2 * j] << 16, d[2 * j] & 0xffff0000u));
                    v[2 * j + 1] = mul2(make_float2(a.scale * e.z, a.scale * e.w), f2(d[2 * j + 1] << 16, d[2 * j + 1] & 0xffff0000u));
                }
                put_parts(at + kColW + 16 * half, 32, v);
            }
            tmem_put_wait();
            tc_fence_before();
            mbar_arrive(w_ready);
            ok = mbar_wait_warp(u_full, ph, wc);
            if (!ok) break;
            tc_fence_after();
            {
                uint32_t x[32];
                float2 v[16];
                tmem_ld32(at + kColX + 32 * half, x);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float4 e = four(g.eG, j), b = four(g.beta, j);
                    v[2 * j] = mul2(make_float2(-b.x * e.x, -b.y * e.y), f2(x[4 * j], x[4 * j + 1]));
                    v[2 * j + 1] = mul2(make_float2(-b.z * e.z, -b.w * e.w), f2(x[4 * j + 2], x[4 * j + 3]));
                }
                put_parts(at + kColZ + 16 * half, 32, v);
                tmem_put_wait();
                tc_fence_before();
                mbar_arrive(z_ready);
                const int rows = ch.n - 32 * half;
                const int64_t stride = (int64_t)a.Hv * kD;
                bf16 *o = static_cast<bf16 *>(a.dv_) + ((int64_t)(ch.tok0 + 32 * half) * a.Hv + h) * kD + m;
                float *r = a.dr + (cell * C + 32 * half) * kD + m;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float4 b = four(g.beta, j);
                    const float bb[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float y = __uint_as_float(x[4 * j + e]);
                        r[(4 * j + e) * kD] = y;
                        if (4 * j + e < rows) o[e * stride] = __float2bfloat16_rn(bb[e] * y);
                    }
                    o += 4 * stride;
                }
            }
            const float2 eC = make_float2(g.eC, g.eC);
            __syncwarp();
            if (lane == 0) mbar_arrive(g_empty + s);
            if (i + 1 < n_chunks) {
                take(i + 1);
                if (!ok) break;
            }
            ok = mbar_wait_warp(d_full, ph, wc);
            if (!ok) break;
            tc_fence_after();
            {
                uint32_t x[64];
                tmem_ld64(at + kColD + 64 * half, x);
#pragma unroll
                for (int j = 0; j < 32; ++j) S[j] = fma2(eC, S[j], f2(x[2 * j], x[2 * j + 1]));
            }
        }
        if (ok && !bad && a.dstate0) {
#pragma unroll
            for (int j = 0; j < 32; ++j) {
                a.dstate0[place + 2 * j * kD] = S[j].x;
                a.dstate0[place + (2 * j + 1) * kD] = S[j].y;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 2) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

__global__ void __launch_bounds__(kThreads, 1) delta_tc_scan_kernel(const __grid_constant__ ScanParams p) {
    scan_body<false>(p, blockIdx.x);
}
// The backward's two walks need nothing of each other, and each is bound by its longest chain, which leaves SMs idle: one
// launch of both (8192 tokens of 16 heads in 7 documents: 254 and 285 us one behind the other, 304 so).  Blocks of one
// walk come 16 in a row, the longest first: neighbouring SMs share an instruction cache that does not hold both walks
// (blocks in turn: 502 us).
constexpr int kTurn = 16;
__global__ void __launch_bounds__(kThreads, 1) delta_tc_walks_kernel(const __grid_constant__ ScanParams p) {
    const int turn = blockIdx.x / kTurn, i = turn / 2 * kTurn + blockIdx.x % kTurn;
    if (i >= p.a.N * p.a.Hv) return;
    if (turn & 1)
        scan_body<true>(p, i);
    else
        back_body(p, i);
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    });
    return fn;
}

// kernel: one of the walks.
template <void (*kernel)(const ScanParams)>
cudaError_t walk(const ScanParams &p, int blocks, cudaStream_t st) {
    static std::atomic<bool> ready[128] = {};
    static_assert(kSmem <= 232448 - 2 * sizeof(Gates), "shared memory of one CTA");
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 128 || !ready[dev]) {
        e = cudaFuncSetAttribute((const void *)kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e != cudaSuccess) return e;
        // The register split draws on the 384 x 168 of the launch: with fewer, the increase could never be granted.
        cudaFuncAttributes fa;
        e = cudaFuncGetAttributes(&fa, (const void *)kernel);
        if (e != cudaSuccess) return e;
        if (fa.numRegs < 168) return cudaErrorInvalidConfiguration;
        if (dev >= 0 && dev < 128) ready[dev] = true;
    }
    return launch_next(kernel, dim3((unsigned)blocks), kThreads, kSmem, st, p);
}

}  // namespace

// Rows [T][H][128] of bf16, `stride` elements apart, in boxes of 64 tokens of one head: 64 columns wide with the
// tensor cores' swizzle, or 128 without.
bool delta_rows_map(CUtensorMap *m, const void *x, int64_t T, int H, int64_t stride, bool swizzle) {
    auto fn = encode_fn();
    if (!fn) return false;
    if (T == 1) stride = (int64_t)H * kD;  // (a single row has no stride)
    const cuuint64_t dims[3] = {kD, (cuuint64_t)H, (cuuint64_t)T}, strides[2] = {kD * 2, (cuuint64_t)stride * 2};
    const cuuint32_t box[3] = {swizzle ? 64u : 128u, 1, C}, es[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(x), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool delta_tc_supported(const DeltaArgs &a) { return delta_tc_shape(a.dtype == RA_BF16, a.dk, a.dv) && a.T > 0; }

cudaError_t launch_delta_tc_scan(const DeltaArgs &a, cudaStream_t st) {
    ScanParams p;
    memset(&p, 0, sizeof(p));
    if (!delta_rows_map(&p.tmQ, a.q, a.T, a.Hk, a.q_stride, true) || !delta_rows_map(&p.tmK, a.k, a.T, a.Hk, a.k_stride, true) ||
        !delta_rows_map(&p.tmV, a.v, a.T, a.Hv, a.v_stride, false))
        return cudaErrorInvalidValue;
    p.a = a;
    p.budget_ns = wait_budget_ns();
    return walk<delta_tc_scan_kernel>(p, a.N * a.Hv, st);
}

cudaError_t launch_delta_tc_walks(const DeltaArgs &a, cudaStream_t st) {
    ScanParams p;
    memset(&p, 0, sizeof(p));
    if (!delta_rows_map(&p.tmQ, a.q, a.T, a.Hk, a.q_stride, true) || !delta_rows_map(&p.tmK, a.k, a.T, a.Hk, a.k_stride, true) ||
        !delta_rows_map(&p.tmV, a.v, a.T, a.Hv, a.v_stride, false) || !delta_rows_map(&p.tmO, a.dout, a.T, a.Hv, a.dout_stride, false))
        return cudaErrorInvalidValue;
    p.a = a;
    p.budget_ns = wait_budget_ns();
    return walk<delta_tc_walks_kernel>(p, (a.N * a.Hv + kTurn - 1) / kTurn * 2 * kTurn, st);
}

}  // namespace ra

// ra_delta_tc_grads.cu -- the gated delta rule's gradients within a chunk on the
// 5th-generation tensor cores (bf16, heads of 128), from what the two walks of
// ra_delta_tc.cu left; the formulas are in ra_delta_bwd.cu.
//
// Bound: a chunk and head reads 270 KB (two states, u, r and dR in fp32; q, k and
// do) and takes about 9000 cycles of products, parts and all, of 27,000 (8192
// tokens, 16 heads: 211 us, 2.6 TB/s); eleven products
// share their operands, so those are made once, in shared memory:
//  * for each half of v: S0, dS1 (rows of dk) and u, dR (rows of tokens) as three
//    bf16 parts; then, with dk as rows of the result (a TMEM lane each),
//      [B' | Q'] = S0 [dR | do]^T,  F' = dS1 u^T,
//    and with the tokens of dR and of do as rows, P' = [dR; do] u^T;
//  * from P', a row a thread: dP, W = -D o (dR u^T) and M = beta W as parts;
//  * dP K, dP^T Q + M^T K and W K, again with dk as rows.
// A token's sums over dk then are sums over lanes: dG_i = q_i.dq_i
// - k_i.(dP^T Q + M^T K + F)_i + k_i.(M K + B)_i needs no sums of P's rows and
// columns, and dbeta_i = dR_i.r_i + k_i.(W K)_i.
// Persistent CTAs, one a SM, take a chunk's value heads of one key head one behind
// the other and sum their dq and dk in TMEM.  Every wait is bounded, and what a thread finds of
// one is agreed on by all before the next barrier.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstring>

#include "ra_delta.cuh"
#include "ra_delta_maps.h"
#include "ra_internal.h"
#include "ra_serve.cuh"

namespace ra {
namespace {

using namespace delta;

constexpr int kThreads = 512;
constexpr int kD = 128, kNP = 3;
constexpr uint32_t kHalf = 16384, kQuarter = 8192;  // 128, 64 rows of 128 bytes
constexpr uint32_t kOffKQ = 0;                      // [2 halves of dk][K's 64 rows, Q's 64 rows]
constexpr uint32_t kOffRD = kOffKQ + 2 * kHalf;     // [2 halves of v][dR's first part, do]
constexpr uint32_t kOffR = kOffRD + 2 * kHalf;      // [2 further parts of dR][64 rows, 64 rows of zeros], of one half of v
constexpr uint32_t kOffU = kOffR + 2 * kHalf;       // [3 parts of u], of one half of v
constexpr uint32_t kOffS = kOffU + 3 * kQuarter;    // [S0, dS1][3 parts], of one half of v
constexpr uint32_t kOffSq = kOffS;                  // [dP, W, M][3 parts], when the products above are done
constexpr uint32_t kOffBar = kOffS + 6 * kHalf;
constexpr uint32_t kSmem = kOffBar + 64 + 1024;
constexpr int kColB = 0, kColQ = 64, kColF = 128, kColP = 192, kColQ2 = 192, kColA2 = 320, kColB2 = 384;  // (P' is read when Q2 is made)
constexpr int kColSumQ = 256, kColSumK = 448;  // dq and dk of a key head's value heads so far

struct GradParams {
    CUtensorMap tmQ, tmK, tmO;
    DeltaArgs a;
    unsigned long long budget_ns;
};

struct Shared {
    Gates g;
    float red[2][4][C];  // of dG and of dbeta: a token's sums over a warp's lanes
    float rr[C], far[16], ss[16];
};

__device__ __forceinline__ uint32_t swz(int row, int byte) { return row * 128 + ((((byte >> 4) ^ row) & 7) << 4) + (byte & 15); }
// Four neighbouring floats of a row into parts, `apart` bytes from each other.
__device__ __forceinline__ void put4(uint8_t *tile, int row, int col, float4 x, const uint32_t (&part)[kNP]) {
    const uint32_t at = swz(row, col * 2);
#pragma unroll
    for (int p = 0; p < kNP; ++p) {
        const uint32_t a = pack_bf16x2(x.x, x.y), b = pack_bf16x2(x.z, x.w);
        *reinterpret_cast<uint2 *>(tile + part[p] + at) = make_uint2(a, b);
        x.x -= __uint_as_float(a << 16), x.y -= __uint_as_float(a & 0xffff0000u);
        x.z -= __uint_as_float(b << 16), x.w -= __uint_as_float(b & 0xffff0000u);
    }
}
// 16 neighbouring floats of a square's row, from column 16 c on, into its parts.
__device__ __forceinline__ void put16(uint8_t *square, int row, int c, float (&x)[16]) {
#pragma unroll
    for (int p = 0; p < kNP; ++p) {
        uint32_t h[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            h[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
            x[2 * i] -= __uint_as_float(h[i] << 16);
            x[2 * i + 1] -= __uint_as_float(h[i] & 0xffff0000u);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
            *reinterpret_cast<uint4 *>(square + p * kQuarter + swz(row, 32 * c + 16 * i)) =
                make_uint4(h[4 * i], h[4 * i + 1], h[4 * i + 2], h[4 * i + 3]);
    }
}
// The sum over the warp's lanes of x[i], in lanes i and i + 16.
__device__ __forceinline__ float lane_sums(float (&x)[16]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 8; o; o >>= 1)
#pragma unroll
        for (int i = 0; i < o; ++i) {
            const bool up = lane & o;
            const float send = up ? x[i] : x[i + o], stay = up ? x[i + o] : x[i];
            x[i] = stay + __shfl_xor_sync(0xffffffffu, send, o);
        }
    return x[0] + __shfl_xor_sync(0xffffffffu, x[0], 16);
}
// TMEM -> registers: 16 columns.
__device__ __forceinline__ void tmem_ld16(uint32_t a, uint32_t (&x)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;\n"
        : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]), "=r"(x[4]), "=r"(x[5]), "=r"(x[6]), "=r"(x[7]), "=r"(x[8]), "=r"(x[9]), "=r"(x[10]), "=r"(x[11]), "=r"(x[12]), "=r"(x[13]), "=r"(x[14]), "=r"(x[15])
        : "r"(a)
        : "memory");
}

__global__ void __launch_bounds__(kThreads, 1) delta_tc_grads_kernel(const __grid_constant__ GradParams p) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ Shared sh;
    const DeltaArgs &a = p.a;
    const uint32_t raw_s = smem_u32(smem_raw), base_s = (raw_s + 1023u) & ~1023u;
    uint8_t *base = smem_raw + (base_s - raw_s);
    uint64_t *bars = reinterpret_cast<uint64_t *>(base + kOffBar);
    uint64_t *full = bars + 0, *done = bars + 1;  // rows landed; products done
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 2);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(bars + 3);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        *abort_flag = 0;
        mbar_init(full, 1);
        mbar_init(done, 1);
        fence_mbar_init();
        tma_prefetch_desc(&p.tmQ);
        tma_prefetch_desc(&p.tmK);
        tma_prefetch_desc(&p.tmO);
    }
    if (warp == 0) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    for (int i = tid; i < 2 * (int)kQuarter / 16; i += kThreads)  // (the rows of zeros)
        *reinterpret_cast<uint4 *>(base + kOffR + (i / 512) * kHalf + kQuarter + i % 512 * 16) = make_uint4(0, 0, 0, 0);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const WaitCtl wc{abort_flag, a.status, p.budget_ns};
    const uint32_t id128 = idesc_bf16_f32(128, 128, 0, 0), id64 = idesc_bf16_f32(128, 64, 0, 0),
                   id64a = idesc_bf16_f32(128, 64, 1, 0), id64ab = idesc_bf16_f32(128, 64, 1, 1);
    uint32_t n_done = 0, n_full = 0;
    bool ok = true;
    wait_ahead();
    const int share = a.Hv / a.Hk;
    const int64_t units = (int64_t)a.hdr->chunks * a.Hk;
    const int quad = warp & 3, part = warp >> 2;  // 32 lanes, 16 tokens
    const uint32_t at = tmem + ((uint32_t)(quad * 32) << 16);
    int turn = 0;  // of the key head's value heads
    for (int64_t unit = blockIdx.x; unit < units; turn = turn + 1 == share ? 0 : turn + 1, unit += turn ? 0 : gridDim.x) {
        const int c = (int)(unit / a.Hk), hk = (int)(unit - (int64_t)c * a.Hk), h = hk * share + turn;
        const int64_t cell = (int64_t)c * a.Hv + h;
        const DeltaChunk ch = a.chunk[c];
        if (tid == 0) {
            mbar_arrive_expect_tx(full, 6 * kQuarter);
            for (int d = 0; d < 2; ++d) {
                tma_load_3d(base + kOffKQ + d * kHalf, &p.tmK, full, d * 64, hk, ch.tok0);
                tma_load_3d(base + kOffKQ + d * kHalf + kQuarter, &p.tmQ, full, d * 64, hk, ch.tok0);
                tma_load_3d(base + kOffRD + d * kHalf + kQuarter, &p.tmO, full, d * 64, h, ch.tok0);
            }
        }
        if (warp == 15) {
            float g[2], b[2];
            gates_load(a, ch, h, g, b);
            gates_put(sh.g, g, b);
        }
        float ss = 0.f, rr[2] = {0.f, 0.f};
        const uint32_t parts_s[kNP] = {0, kHalf, 2 * kHalf}, parts_u[kNP] = {0, kQuarter, 2 * kQuarter};
#pragma unroll 1
        for (int v = 0; v < 2 && ok; ++v) {
            // this half's rows, all on their way at once (and beside the last half's products)
            float4 s0[4], ds[4], u[2], dr[2], r[2];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int64_t x = (cell * kD + (tid >> 4) + 32 * e) * kD + 64 * v + (tid & 15) * 4;
                s0[e] = __ldcs(reinterpret_cast<const float4 *>(a.s0 + x));
                ds[e] = __ldcs(reinterpret_cast<const float4 *>(a.ds + x));
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int64_t x = (cell * C + (tid >> 4) + 32 * e) * kD + 64 * v + (tid & 15) * 4;
                u[e] = __ldcs(reinterpret_cast<const float4 *>(a.u + x));
                dr[e] = __ldcs(reinterpret_cast<const float4 *>(a.dr + x));
                r[e] = __ldcs(reinterpret_cast<const float4 *>(a.r + x));
            }
            if (v) {
                ok = mbar_wait(done, n_done++ & 1u, wc);
                ok = __syncthreads_and(ok);
                if (!ok) break;
                tc_fence_after();
            }
            const uint32_t parts_r[kNP] = {kOffRD + v * kHalf, kOffR, kOffR + kHalf};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                ss += s0[e].x * ds[e].x + s0[e].y * ds[e].y + s0[e].z * ds[e].z + s0[e].w * ds[e].w;
                put4(base + kOffS, (tid >> 4) + 32 * e, (tid & 15) * 4, s0[e], parts_s);
                put4(base + kOffS + 3 * kHalf, (tid >> 4) + 32 * e, (tid & 15) * 4, ds[e], parts_s);
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                rr[e] += dr[e].x * r[e].x + dr[e].y * r[e].y + dr[e].z * r[e].z + dr[e].w * r[e].w;
                put4(base + kOffU, (tid >> 4) + 32 * e, (tid & 15) * 4, u[e], parts_u);
                put4(base, (tid >> 4) + 32 * e, (tid & 15) * 4, dr[e], parts_r);
            }
            if (v == 0) {
                ok = mbar_wait(full, n_full++ & 1u, wc);
                if (ch.n < C && ok)  // rows of K, Q and do behind the sequence's end are another's, or none
                    for (int i = tid; i < 6 * (C - ch.n) * 8; i += kThreads) {
                        const int t = i / ((C - ch.n) * 8), x = i % ((C - ch.n) * 8);
                        uint8_t *tile = base + (t < 4 ? kOffKQ + t * kQuarter : kOffRD + (t - 4) * kHalf + kQuarter);
                        *reinterpret_cast<uint4 *>(tile + (ch.n * 8 + x) * 16) = make_uint4(0, 0, 0, 0);
                    }
            }
            fence_proxy_async_smem();
            ok = __syncthreads_and(ok);
            if (!ok) break;
            if (warp == 0) {
                tc_fence_after();  // (behind the last cell's reads of what these products write over)
                const uint64_t dS = sdesc_sw128(base_s + kOffS, 16, 1024), dD = sdesc_sw128(base_s + kOffS + 3 * kHalf, 16, 1024);
                const uint64_t dRD = sdesc_sw128(base_s + kOffRD + v * kHalf, 16, 1024), dR = sdesc_sw128(base_s + kOffR, 16, 1024);
                const uint64_t dU = sdesc_sw128(base_s + kOffU, 16, 1024);
                // A's part i by B's part j, 64 columns of v: four products
                auto four = [&](uint32_t d, uint64_t x, uint64_t y, uint32_t id, bool first) {
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks) tc_mma_ss(tmem + d, x + 2 * ks, y + 2 * ks, id, !(first && ks == 0));
                };
                auto S = [&](uint64_t x, int i) { return x + (uint32_t)i * (kHalf >> 4); };
                auto U = [&](int j) { return dU + (uint32_t)j * (kQuarter >> 4); };
                auto R = [&](int i) { return i ? S(dR, i - 1) : dRD; };  // (dR's part i; with do's rows behind the first)
                if (elected()) {  // (one thread for all of them: an issue takes less than a product)
                    four(kColB, S(dS, 2), dRD, id128, v == 0);
                    four(kColB, S(dS, 1), dRD, id128, false);
                    four(kColB, S(dS, 1), R(1), id64, false);
                    four(kColB, S(dS, 0), R(2), id64, false);
                    four(kColB, S(dS, 0), R(1), id64, false);
                    four(kColB, S(dS, 0), dRD, id128, false);
#pragma unroll
                    for (int o = 2; o >= 0; --o)
#pragma unroll
                        for (int i = 0; i <= o; ++i) {
                            four(kColF, S(dD, i), U(o - i), id64, v == 0 && o == 2 && i == 0);
                            four(kColP, R(i), U(o - i), id64, v == 0 && o == 2 && i == 0);
                        }
                }
                __syncwarp();
                tc_commit_w(done);
            }
        }
        if (!ok) break;
        // dP, W and M from the rows of P'
        ok = mbar_wait(done, n_done++ & 1u, wc);
        ok = __syncthreads_and(ok);
        if (!ok) break;
        tc_fence_after();
        {
            const int row = quad * 32 + lane, i = row & 63;  // lanes 0 to 63: dR u^T, 64 to 127: do u^T
            const bool w = quad < 2;
            uint32_t x[16];
            float y[16];
            tmem_ld16(at + kColP + 16 * part, x);
            const float f = w ? -1.f : a.scale;
            const float2 me = make_float2(sh.g.hi[i], sh.g.lo[i]);
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const int t = 16 * part + j;
                const float D = gate_exp(me, make_float2(sh.g.hi[t], sh.g.lo[t]));
                y[j] = t + (w ? 1 : 0) <= i ? f * D * __uint_as_float(x[j]) : 0.f;
            }
            uint8_t *sq = base + kOffSq;
            if (w) {
                float z[16];
                const float b = sh.g.beta[i];
#pragma unroll
                for (int j = 0; j < 16; ++j) z[j] = b * y[j];
                put16(sq + 3 * kQuarter, i, part, y);
                put16(sq + 6 * kQuarter, i, part, z);
            } else {
                put16(sq, i, part, y);
            }
        }
        tc_fence_before();
        fence_proxy_async_smem();
        __syncthreads();
        if (warp == 0) {
            tc_fence_after();
            const uint64_t K = sdesc_sw128(base_s + kOffKQ, kHalf, 1024), Q = sdesc_sw128(base_s + kOffKQ + kQuarter, kHalf, 1024);
            // 64 tokens' rows of K or Q, their dk as rows of the result, by a square's parts (rows: `rows` bytes to the next 16)
            auto by = [&](uint32_t d, uint64_t x, uint32_t square, uint32_t lbo, uint32_t step, uint32_t id, bool first) {
                const uint64_t s = sdesc_sw128(base_s + kOffSq + square * 3 * kQuarter, lbo, 1024);
#pragma unroll
                for (int q = kNP - 1; q >= 0; --q)
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
                        tc_mma_ss(tmem + d, x + ((uint32_t)ks * 2048u >> 4), s + (((uint32_t)q * kQuarter + (uint32_t)ks * step) >> 4), id,
                                    !(first && q == kNP - 1 && ks == 0));
            };
            if (elected()) {
                by(kColQ2, K, 0, 16, 32, id64a, true);
                by(kColA2, Q, 0, kHalf, 2048, id64ab, true);
                by(kColA2, K, 2, kHalf, 2048, id64ab, false);
                by(kColB2, K, 1, 16, 32, id64a, true);
            }
            __syncwarp();
            tc_commit_w(done);
        }
        // beside them: the next cell's way to L2, a line of 128 bytes a thread and turn (without it the gradients of 8192
        // tokens take 588 us in place of 564); and sums of what was loaded
        const int64_t next_unit = turn + 1 < share ? unit : unit + gridDim.x;
        if (next_unit < units) {
            const int64_t next = next_unit * share + (turn + 1 < share ? turn + 1 : 0);  // (units and cells are in one order)
            auto fetch = [&](const float *x, int floats) {
                for (int i = tid * 32; i < floats; i += kThreads * 32) asm volatile("prefetch.global.L2 [%0];" ::"l"(x + next * floats + i));
            };
            fetch(a.s0, kD * kD);
            fetch(a.ds, kD * kD);
            fetch(a.u, C * kD);
            fetch(a.dr, C * kD);
            fetch(a.r, C * kD);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int o = 1; o < 16; o <<= 1) rr[e] += __shfl_xor_sync(0xffffffffu, rr[e], o);
            if ((tid & 15) == 0) sh.rr[(tid >> 4) + 32 * e] = rr[e];
        }
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (lane == 0) sh.ss[warp] = ss;
        ok = mbar_wait(done, n_done++ & 1u, wc);
        ok = __syncthreads_and(ok);
        if (!ok) break;
        tc_fence_after();
        {
            const int m = quad * 32 + lane;  // dk
            float far = 0.f, sum[16], db[16];
            const uint8_t *kq = base + kOffKQ + (m >> 6) * kHalf;
            const int64_t stride = (int64_t)a.Hk * kD, o0 = ((int64_t)(ch.tok0 + 16 * part) * a.Hk + hk) * kD + m;
            const int rows = ch.n - 16 * part;
            // a gradient of this head: to the sums, or with them to the tensor
            auto put = [&](uint32_t col, float (&x)[16], void *to) {
                if (turn > 0) {
                    uint32_t s[16];
                    tmem_ld16(at + col + 16 * part, s);
#pragma unroll
                    for (int j = 0; j < 16; ++j) x[j] += __uint_as_float(s[j]);
                }
                if (turn + 1 < share) {
                    uint32_t s[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) s[j] = __float_as_uint(x[j]);
                    tmem_st16(at + col + 16 * part, s);
                    return;
                }
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    if (j < rows) static_cast<bf16 *>(to)[o0 + j * stride] = __float2bfloat16_rn(x[j]);
            };
            auto value = [&](int row) {
                return __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t *>(kq + swz(row, (m & 63) * 2)) << 16);
            };
            uint32_t x[16], y[16];
            tmem_ld16x2(at + kColQ + 16 * part, at + kColQ2 + 16 * part, x, y);
            float dq[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const int t = 16 * part + j;
                dq[j] = fmaf(a.scale * sh.g.eG[t], __uint_as_float(x[j]), __uint_as_float(y[j]));
                sum[j] = value(C + t) * dq[j];
            }
            put(kColSumQ, dq, a.dq);
            tmem_ld16x2(at + kColF + 16 * part, at + kColA2 + 16 * part, x, y);
            float dk[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const int t = 16 * part + j;
                const float k = value(t), F = sh.g.eL[t] * __uint_as_float(x[j]);
                far += F * k;
                dk[j] = F + __uint_as_float(y[j]);
                sum[j] -= k * dk[j];
            }
            tmem_ld16x2(at + kColB + 16 * part, at + kColB2 + 16 * part, x, y);
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const int t = 16 * part + j;
                const float k = value(t), W = __uint_as_float(y[j]);
                const float b = sh.g.beta[t] * fmaf(-sh.g.eG[t], __uint_as_float(x[j]), W);
                db[j] = k * W;
                sum[j] += k * b;
                dk[j] += b;
            }
            put(kColSumK, dk, a.dk_);
            tc_fence_before();
            const float r0 = lane_sums(sum), r1 = lane_sums(db);
            if (lane < 16) {
                sh.red[0][quad][16 * part + lane] = r0;
                sh.red[1][quad][16 * part + lane] = r1;
            }
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) far += __shfl_xor_sync(0xffffffffu, far, o);
            if (lane == 0) sh.far[warp] = far;
        }
        __syncthreads();
        if (warp == 0) {  // the gates: sums from each token to the chunk's end
            float end = 0.f, s = 0.f, x[2];
#pragma unroll
            for (int w = 0; w < 16; ++w) {
                end += sh.far[w];
                s += sh.ss[w];
            }
            end += s * sh.g.eC;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int t = 2 * lane + e;
                x[e] = (sh.red[0][0][t] + sh.red[0][1][t]) + (sh.red[0][2][t] + sh.red[0][3][t]);
                const float b = (sh.red[1][0][t] + sh.red[1][1][t]) + (sh.red[1][2][t] + sh.red[1][3][t]);
                if (t < ch.n) a.dbeta[(int64_t)(ch.tok0 + t) * a.Hv + h] = sh.rr[t] + b;
            }
            float sum = x[0] + x[1];  // of this lane's tokens and all behind
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const float y = __shfl_down_sync(0xffffffffu, sum, o);
                if (lane + o < 32) sum += y;
            }
            const float y = __shfl_down_sync(0xffffffffu, sum, 1), after = lane < 31 ? y : 0.f;
            const int64_t o = (int64_t)(ch.tok0 + 2 * lane) * a.Hv + h;
            if (2 * lane < ch.n) a.dg[o] = sum + end;
            if (2 * lane + 1 < ch.n) a.dg[o + a.Hv] = x[1] + after + end;
        }
        __syncthreads();  // (the gates and sums are read, and every product is done)
    }
    if (!ok) {
        // copies and products under way must have ended before the CTA may
        volatile int local_abort = 0;
        const WaitCtl drain{&local_abort, a.status, p.budget_ns};
        if (warp == 0) {
            tc_commit_w(done);
            (void)mbar_wait(done, n_done & 1u, drain);
        }
        if (tid == 0) (void)mbar_wait(full, n_full & 1u, drain);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

}  // namespace

cudaError_t launch_delta_tc_grads(const DeltaArgs &a, cudaStream_t st) {
    GradParams p;
    memset(&p, 0, sizeof(p));
    if (!delta_rows_map(&p.tmQ, a.q, a.T, a.Hk, a.q_stride, true) || !delta_rows_map(&p.tmK, a.k, a.T, a.Hk, a.k_stride, true) ||
        !delta_rows_map(&p.tmO, a.dout, a.T, a.Hv, a.dout_stride, true))
        return cudaErrorInvalidValue;
    p.a = a;
    p.budget_ns = wait_budget_ns();
    static LaunchFit fit;
    static_assert(kSmem + sizeof(Shared) <= 232448, "shared memory of one CTA");
    const cudaError_t e = fit.prepare(reinterpret_cast<const void *>(delta_tc_grads_kernel), kThreads, kSmem, nullptr);
    if (e != cudaSuccess) return e;
    return launch_next(delta_tc_grads_kernel, dim3(paged_sms()), kThreads, kSmem, st, p);
}

}  // namespace ra

// ra_delta_bwd.cu -- gradients of the gated delta rule.
//
// With the forward's formulas (ra_delta.cu), the state S0 ahead of each chunk,
// u and r kept by a forward walk, and dS1 the gradient of the state behind a
// chunk:
//   du = e^(G_63 - G) (K dS1) + P^T do,   dR = T^T du,   dv = beta dR
//   dS0 = e^(G_63) dS1 + Q^T (scale e^G do) - K^T (beta e^G dR)
// is a walk over each sequence's chunks from its end, like the forward's.  All
// else needs a chunk's own rows and the two states, and is done for all chunks
// at once:
//   dP_ij = scale D_ij do_i.u_j (j <= i),   M_ij = -beta_i D_ij dR_i.u_j (j < i)
//   dq = scale e^G (do S0^T) + dP K
//   dk = dP^T Q + (M + M^T) K + F + B,
//        F = e^(G_63 - G) (u dS1^T),  B = -beta e^G (dR S0^T)
//   dbeta_i = dR_i.r_i - sum_j D_ij (dR_i.u_j) (k_i.k_j)
//   dG_i = sum_j (E_ij - E_ji) + scale e^G_i (do_i S0^T).q_i + B_i.k_i - F_i.k_i,
//        E = dP (q.k) + M (k.k)
//   dg_t = sum over i >= t of dG_i, + sum F.k + e^(G_63) <S0, dS1>
#include <cuda_bf16.h>
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include "ra_delta.cuh"
#include "ra_serve.cuh"

namespace ra {
namespace {

namespace cg = cooperative_groups;

using namespace delta;

constexpr int kThreads = 256;

// ------------------------------------------------------------ the walk from the end
template <typename E, int DK, int DVS>
struct BackSmem {
    static constexpr bool F = std::is_same<E, float>::value;
    static constexpr int NPI = F ? 3 : 1, KB = F ? 1 : 2, LD = DK + 8, LV = DVS + 8;
    bf16 k[KB][NPI][C][LD], q[NPI][C][LD];
    bf16 T[NP][C][kLdc], P[NP][C][kLdc];
    bf16 S[NP][DK][LV];   // dS1
    bf16 X[NP][C][LV];    // du, then scale e^G do
    bf16 Y[NP][C][LV];    // do, then -beta e^G dR
    Gates g[2];
};

template <typename E, int DK, int DVS>
__global__ void __launch_bounds__(kThreads, 1) delta_back_kernel(const DeltaArgs a) {
    using Smem = BackSmem<E, DK, DVS>;
    constexpr int NPI = Smem::NPI, KB = Smem::KB, LD = Smem::LD, LV = Smem::LV;
    constexpr int MW = DK / 16, NS = DVS / 8 / (8 / MW), NX = DVS / 16;
    constexpr int PK = C * LD * 2, PT = C * kLdc * 2, PS = DK * LV * 2, PR = C * LV * 2;
    extern __shared__ __align__(128) uint8_t raw[];
    Smem &sm = *reinterpret_cast<Smem *>(raw);
    wait_ahead();
    if (a.hdr->bad) return;
    const int slices = a.dv / DVS, per = a.Hv * slices;
    const int seq = a.order[blockIdx.x / per], h = blockIdx.x % per / slices, v0 = blockIdx.x % slices * DVS;
    const int hk = h / (a.Hv / a.Hk), dv = a.dv;
    const int c0 = a.first[seq], c1 = a.first[seq + 1];
    const int tid = threadIdx.x, warp = tid >> 5;
    const int srow = 16 * (warp % MW), scol = warp / MW * 8 * NS;
    const int xrow = 16 * (warp & 3), xcol = (warp >> 2) * 8 * NX;
    const int64_t splace = ((int64_t)seq * a.Hv + h) * DK * dv + v0;

    float S[NS][4];
#pragma unroll
    for (int n = 0; n < NS; ++n)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            float2 x = make_float2(0.f, 0.f);
            if (a.dstate)
                x = *reinterpret_cast<const float2 *>(a.dstate + splace + (int64_t)(srow + acc_row(hf)) * dv + scol + acc_col(n));
            S[n][2 * hf] = x.x;
            S[n][2 * hf + 1] = x.y;
        }
    auto load_k = [&](int c, int buf) {
        const DeltaChunk ch = a.chunk[c];
        load_rows<E, DK, kThreads>(&sm.k[buf][0][0][0], LD, C * LD, static_cast<const E *>(a.k) + ch.tok0 * a.k_stride + hk * DK,
                                   a.k_stride, ch.n);
    };
    auto load_q = [&](int c) {
        const DeltaChunk ch = a.chunk[c];
        load_rows<E, DK, kThreads>(&sm.q[0][0][0], LD, C * LD, static_cast<const E *>(a.q) + ch.tok0 * a.q_stride + hk * DK,
                                   a.q_stride, ch.n);
    };
    auto load_tp = [&](int c, int which) {
        load_square<NP, kThreads>(which ? &sm.P[0][0][0] : &sm.T[0][0][0],
                                  a.tp + (((int64_t)c * a.Hv + h) * 2 + which) * NP * C * C);
    };
    float gg[2], gb[2];
    if (c0 < c1) {
        if (KB == 2) load_k(c1 - 1, 0);
        load_tp(c1 - 1, 1);
        cp_commit();
        load_tp(c1 - 1, 0);
        cp_commit();
        if (KB == 2) load_q(c1 - 1);
        cp_commit();
        if (warp == 0) gates_load(a, a.chunk[c1 - 1], h, gg, gb);
    }
    for (int c = c1 - 1; c >= c0; --c) {
        const int at = c1 - 1 - c, buf = KB == 2 ? at & 1 : 0;
        const DeltaChunk ch = a.chunk[c];
        Gates &g = sm.g[at & 1];
        const int64_t cell = (int64_t)c * a.Hv + h;
        __syncthreads();  // (the last chunk's products with Q, K, X and Y)
        if (KB == 1) {
            load_k(c, 0);
            load_q(c);
        }
        if (at) {
            if (KB == 2) load_q(c);
            cp_commit();
        }
        if (warp == 0) {
            gates_put(g, gg, gb);
            if (c > c0) gates_load(a, a.chunk[c - 1], h, gg, gb);
        }
        float2 d[NX][2];
#pragma unroll
        for (int n = 0; n < NX; ++n)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const int i = xrow + acc_row(hf), j = xcol + acc_col(n);
                d[n][hf] = make_float2(0.f, 0.f);
                if (i < ch.n)
                    d[n][hf] = load2(static_cast<const E *>(a.dout) + (ch.tok0 + i) * a.dout_stride + h * dv + v0 + j);
                put2<NPI>(&sm.Y[0][i][j], C * LV, d[n][hf].x, d[n][hf].y);
            }
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const int i = srow + acc_row(hf), j = scol + acc_col(n);
                put2<NP>(&sm.S[0][i][j], DK * LV, S[n][2 * hf], S[n][2 * hf + 1]);
                *reinterpret_cast<float2 *>(a.ds + (cell * DK + i) * dv + v0 + j) = make_float2(S[n][2 * hf], S[n][2 * hf + 1]);
            }
        cp_wait<2>();  // K and P (behind them T, Q)
        __syncthreads();
        if (KB == 2 && c > c0) load_k(c - 1, buf ^ 1);
        float x[NX][4];
        zero(x);
        mm<NX, NPI, NP, NP, false, true>(x, smem_u32(sm.k[buf]) + xrow * LD * 2, LD, PK, smem_u32(sm.S) + xcol * 2, LV, PS, 0,
                                         DK);
#pragma unroll
        for (int n = 0; n < NX; ++n)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const float e = g.eL[xrow + acc_row(hf)];
                x[n][2 * hf] *= e;
                x[n][2 * hf + 1] *= e;
            }
        mm<NX, NP, NPI, NP, true, true>(x, smem_u32(sm.P) + xrow * 2, kLdc, PT, smem_u32(sm.Y) + xcol * 2, LV, PR, xrow, C);
#pragma unroll
        for (int n = 0; n < NX; ++n)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf)
                put2<NP>(&sm.X[0][xrow + acc_row(hf)][xcol + acc_col(n)], C * LV, x[n][2 * hf], x[n][2 * hf + 1]);
        cp_wait<1>();  // T (behind it Q)
        __syncthreads();
        if (c > c0) load_tp(c - 1, 1);
        cp_commit();  // (with the next K)
        zero(x);
        mm<NX, NP, NP, NP, true, true>(x, smem_u32(sm.T) + xrow * 2, kLdc, PT, smem_u32(sm.X) + xcol * 2, LV, PR, xrow, C);
        cp_wait<1>();  // Q (behind it the next K and P)
        __syncthreads();
        if (c > c0) load_tp(c - 1, 0);
        cp_commit();
#pragma unroll
        for (int n = 0; n < NX; ++n)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const int i = xrow + acc_row(hf), j = xcol + acc_col(n);
                const float x0 = x[n][2 * hf], x1 = x[n][2 * hf + 1], b = g.beta[i], e = g.eG[i];
                *reinterpret_cast<float2 *>(a.dr + (cell * C + i) * dv + v0 + j) = make_float2(x0, x1);
                if (i < ch.n)
                    store2(static_cast<E *>(a.dv_) + ((int64_t)(ch.tok0 + i) * a.Hv + h) * dv + v0 + j, b * x0, b * x1);
                put2<NP>(&sm.Y[0][i][j], C * LV, -b * e * x0, -b * e * x1);
                put2<NP>(&sm.X[0][i][j], C * LV, a.scale * e * d[n][hf].x, a.scale * e * d[n][hf].y);
            }
        __syncthreads();
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) S[n][i] *= g.eC;
        mm<NS, NPI, NP, NP, true, true>(S, smem_u32(sm.q) + srow * 2, LD, PK, smem_u32(sm.X) + scol * 2, LV, PR, 0, C);
        mm<NS, NPI, NP, NP, true, true>(S, smem_u32(sm.k[buf]) + srow * 2, LD, PK, smem_u32(sm.Y) + scol * 2, LV, PR, 0, C);
    }
    cp_wait<0>();
    if (a.dstate0) {
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf)
                *reinterpret_cast<float2 *>(a.dstate0 + splace + (int64_t)(srow + acc_row(hf)) * dv + scol + acc_col(n)) =
                    make_float2(S[n][2 * hf], S[n][2 * hf + 1]);
    }
}

// ------------------------------------------------------------ the chunks' gradients
constexpr int kVS = 32;  // columns of the states at a time

template <typename E, int DK>
struct GradSmem {
    static constexpr int NPI = std::is_same<E, float>::value ? 3 : 1, LD = DK + 8, LV = kVS + 8;
    bf16 k[NPI][C][LD], q[NPI][C][LD];
    struct Slice {
        bf16 s0[NP][DK][LV], ds[NP][DK][LV];
        bf16 u[NP][C][LV], dr[NP][C][LV], d[NPI][C][LV];
    };
    struct Square {
        bf16 dP[NP][C][kLdc], M[NP][C][kLdc];
    };
    union {
        Slice v;
        Square c;
    };
    Gates g;
    float row[4][C], db[4][C], col[4][C];  // of each group of columns, of each 16 rows
    float rr[C], far[16], ss[8];
};

// R CTAs (a cluster) a cell, 64 / R rows each.  Of two, the second gives the first what its rows have of the first
// one's columns (dP, M) and its sums for the gates; nothing goes the other way, as dP and M are triangular.
template <typename E, int DK, int R>
__global__ void __launch_bounds__(kThreads, 1) delta_grads_kernel(const DeltaArgs a) {
    using Smem = GradSmem<E, DK>;
    constexpr int NPI = Smem::NPI, LD = Smem::LD, LV = Smem::LV;
    constexpr int RT = C / R / 16, CG = 8 / RT;                 // 16 rows a warp, and a CGth of the columns:
    constexpr int NK = DK / 8 / CG, NC = C / 8 / CG;            // n-tiles along dk, along the chunk
    constexpr int PK = C * LD * 2, PT = C * kLdc * 2, PS = DK * LV * 2, PR = C * LV * 2;
    extern __shared__ __align__(128) uint8_t raw[];
    Smem &sm = *reinterpret_cast<Smem *>(raw);
    const int c = blockIdx.x / R, rank = blockIdx.x % R, h = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    wait_ahead();
    if (c >= a.hdr->chunks) return;
    const DeltaChunk ch = a.chunk[c];
    const int hk = h / (a.Hv / a.Hk), dv = a.dv;
    const int64_t cell = (int64_t)c * a.Hv + h;
    const int row0 = 16 * (rank * RT + warp % RT), group = warp / RT, kcol = group * 8 * NK, ccol = group * 8 * NC;
    auto own = [&](int r) { return R == 1 || r / (C / R) == rank; };
    Smem &first = R == 1 ? sm : *cg::this_cluster().map_shared_rank(&sm, 0);
    auto sync = [&]() {
        if constexpr (R == 1)
            __syncthreads();
        else
            cg::this_cluster().sync();
    };
    load_rows<E, DK, kThreads>(&sm.k[0][0][0], LD, C * LD, static_cast<const E *>(a.k) + ch.tok0 * a.k_stride + hk * DK,
                               a.k_stride, ch.n);
    load_rows<E, DK, kThreads>(&sm.q[0][0][0], LD, C * LD, static_cast<const E *>(a.q) + ch.tok0 * a.q_stride + hk * DK,
                               a.q_stride, ch.n);
    if (warp == 0) {
        float g[2], b[2];
        gates_load(a, ch, h, g, b);
        gates_put(sm.g, g, b);
    }
    float dq[NK][4], F[NK][4], B[NK][4], dP[NC][4], dA[NC][4];
    zero(dq);
    zero(F);
    zero(B);
    zero(dP);
    zero(dA);
    float ss = 0.f;   // <S0, dS1>
    float rr = 0.f;   // dR . r of row tid / 4
    for (int v0 = 0; v0 < dv; v0 += kVS) {
        __syncthreads();
        load_rows<E, kVS, kThreads>(&sm.v.d[0][0][0], LV, C * LV, static_cast<const E *>(a.dout) + ch.tok0 * a.dout_stride + h * dv + v0,
                                    a.dout_stride, ch.n);
        cp_commit();
        for (int i = tid; i < DK * kVS / 4; i += kThreads) {
            const int r = i / (kVS / 4), j = i % (kVS / 4) * 4;
            const float4 x = *reinterpret_cast<const float4 *>(a.s0 + (cell * DK + r) * dv + v0 + j);
            const float4 y = *reinterpret_cast<const float4 *>(a.ds + (cell * DK + r) * dv + v0 + j);
            ss += x.x * y.x + x.y * y.y + x.z * y.z + x.w * y.w;
            put2<NP>(&sm.v.s0[0][r][j], DK * LV, x.x, x.y);
            put2<NP>(&sm.v.s0[0][r][j + 2], DK * LV, x.z, x.w);
            put2<NP>(&sm.v.ds[0][r][j], DK * LV, y.x, y.y);
            put2<NP>(&sm.v.ds[0][r][j + 2], DK * LV, y.z, y.w);
        }
#pragma unroll
        for (int i = 0; i < kVS / 16; ++i) {
            const int r = tid >> 2, j = (tid & 3) * 4 + i * 16;
            const int64_t at = (cell * C + r) * dv + v0 + j;
            const float4 x = *reinterpret_cast<const float4 *>(a.u + at);
            put2<NP>(&sm.v.u[0][r][j], C * LV, x.x, x.y);
            put2<NP>(&sm.v.u[0][r][j + 2], C * LV, x.z, x.w);
            if (!own(r)) continue;
            const float4 y = *reinterpret_cast<const float4 *>(a.dr + at);
            const float4 z = *reinterpret_cast<const float4 *>(a.r + at);
            rr += y.x * z.x + y.y * z.y + y.z * z.z + y.w * z.w;
            put2<NP>(&sm.v.dr[0][r][j], C * LV, y.x, y.y);
            put2<NP>(&sm.v.dr[0][r][j + 2], C * LV, y.z, y.w);
        }
        cp_wait<0>();
        __syncthreads();
        const uint32_t d = smem_u32(sm.v.d) + row0 * LV * 2, u = smem_u32(sm.v.u), dr = smem_u32(sm.v.dr) + row0 * LV * 2;
        const uint32_t s0 = smem_u32(sm.v.s0) + kcol * LV * 2, ds = smem_u32(sm.v.ds) + kcol * LV * 2;
        mm<NK, NPI, NP, NP, false, false>(dq, d, LV, PR, s0, LV, PS, 0, kVS);
        mm<NK, NP, NP, NP, false, false>(F, u + row0 * LV * 2, LV, PR, ds, LV, PS, 0, kVS);
        mm<NK, NP, NP, NP, false, false>(B, dr, LV, PR, s0, LV, PS, 0, kVS);
        mm<NC, NPI, NP, NP, false, false>(dP, d, LV, PR, u + ccol * LV * 2, LV, PR, 0, kVS);
        mm<NC, NP, NP, NP, false, false>(dA, dr, LV, PR, u + ccol * LV * 2, LV, PR, 0, kVS);
    }
    // sums of rows over the four threads that hold them
    rr += __shfl_xor_sync(0xffffffffu, rr, 1);
    rr += __shfl_xor_sync(0xffffffffu, rr, 2);
    if ((tid & 3) == 0) sm.rr[tid >> 2] = rr;
    float row[2] = {0.f, 0.f}, db[2] = {0.f, 0.f}, far = 0.f;
    const uint32_t kb = smem_u32(sm.k), qb = smem_u32(sm.q);
    {
        float kk[NC][4], qk[NC][4];
        zero(kk);
        zero(qk);
        mm<NC, NPI, NPI, 3, false, false>(kk, kb + row0 * LD * 2, LD, PK, kb + ccol * LD * 2, LD, PK, 0, DK);
        mm<NC, NPI, NPI, 3, false, false>(qk, qb + row0 * LD * 2, LD, PK, kb + ccol * LD * 2, LD, PK, 0, DK);
        sync();  // (the slices' products: dP and M take their place)
#pragma unroll
        for (int n = 0; n < NC; ++n) {
            float col[2] = {0.f, 0.f};
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const int i = row0 + acc_row(hf), j = ccol + acc_col(n);
                float p[2], m[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float D = j + e <= i ? decay(sm.g, i, j + e) : 0.f;
                    p[e] = j + e <= i ? a.scale * D * dP[n][2 * hf + e] : 0.f;
                    const float w = j + e < i ? -D * dA[n][2 * hf + e] : 0.f;
                    m[e] = w * sm.g.beta[i];
                    db[hf] += w * kk[n][2 * hf + e];
                    const float x = p[e] * qk[n][2 * hf + e] + m[e] * kk[n][2 * hf + e];
                    row[hf] += x;
                    col[e] += x;
                }
                put2<NP>(&sm.c.dP[0][i][j], C * kLdc, p[0], p[1]);
                put2<NP>(&sm.c.M[0][i][j], C * kLdc, m[0], m[1]);
                if (R > 1 && rank && own(j + C / R)) {
                    put2<NP>(&first.c.dP[0][i][j], C * kLdc, p[0], p[1]);
                    put2<NP>(&first.c.M[0][i][j], C * kLdc, m[0], m[1]);
                }
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) col[e] += __shfl_xor_sync(0xffffffffu, col[e], o);
                if (lane < 4) first.col[row0 / 16][ccol + n * 8 + 2 * lane + e] = col[e];
            }
        }
    }
    // the parts that the states give, and their share of the gates' gradients
#pragma unroll
    for (int n = 0; n < NK; ++n)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            const int i = row0 + acc_row(hf), j = kcol + acc_col(n);
            const float eq = a.scale * sm.g.eG[i], ef = sm.g.eL[i], eb = -sm.g.beta[i] * sm.g.eG[i];
            const float2 k = get2<NPI>(&sm.k[0][i][j], C * LD), q = get2<NPI>(&sm.q[0][i][j], C * LD);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float kx = e ? k.y : k.x, qx = e ? q.y : q.x;
                float &x = dq[n][2 * hf + e], &f = F[n][2 * hf + e];
                const float b = eb * B[n][2 * hf + e];
                x *= eq;
                f *= ef;
                row[hf] += x * qx + b * kx - f * kx;
                far += f * kx;
                f += b;  // dk from here on
            }
        }
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
            row[hf] += __shfl_xor_sync(0xffffffffu, row[hf], o);
            db[hf] += __shfl_xor_sync(0xffffffffu, db[hf], o);
        }
        if ((lane & 3) == 0) {
            first.row[group][row0 + acc_row(hf)] = row[hf];
            sm.db[group][row0 + acc_row(hf)] = db[hf];
        }
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        far += __shfl_xor_sync(0xffffffffu, far, o);
        ss += __shfl_xor_sync(0xffffffffu, ss, o);
    }
    if (lane == 0) {
        first.far[rank * 8 + warp] = far;
        sm.ss[warp] = ss;
    }
    sync();
    if (tid < C && tid < ch.n && own(tid)) {
        float x = sm.rr[tid];
#pragma unroll
        for (int i = 0; i < CG; ++i) x += sm.db[i][tid];
        a.dbeta[(int64_t)(ch.tok0 + tid) * a.Hv + h] = x;
    }
    if (warp == 0 && rank == 0) {  // the gates: sums from each token to the chunk's end
        float end = 0.f, s = 0.f;
#pragma unroll
        for (int w = 0; w < 8 * R; ++w) end += sm.far[w];
#pragma unroll
        for (int w = 0; w < 8; ++w) s += sm.ss[w];
        end += s * sm.g.eC;
        float x[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int t = 2 * lane + e;
            x[e] = 0.f;
#pragma unroll
            for (int i = 0; i < CG; ++i) x[e] += sm.row[i][t];
#pragma unroll
            for (int w = 0; w < 4; ++w) x[e] -= sm.col[w][t];
        }
        float sum = x[0] + x[1];  // of this lane's tokens and all behind
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float y = __shfl_down_sync(0xffffffffu, sum, o);
            if (lane + o < 32) sum += y;
        }
        const float y = __shfl_down_sync(0xffffffffu, sum, 1);
        const float after = lane < 31 ? y : 0.f;
        const int64_t at = (int64_t)(ch.tok0 + 2 * lane) * a.Hv + h;
        if (2 * lane < ch.n) a.dg[at] = sum + end;
        if (2 * lane + 1 < ch.n) a.dg[at + a.Hv] = x[1] + after + end;
    }
    const uint32_t Pb = smem_u32(sm.c.dP), Mb = smem_u32(sm.c.M);
    mm<NK, NP, NPI, NP, false, true>(dq, Pb + row0 * kLdc * 2, kLdc, PT, kb + kcol * 2, LD, PK, 0, row0 + 16);
    mm<NK, NP, NPI, NP, true, true>(F, Pb + row0 * 2, kLdc, PT, qb + kcol * 2, LD, PK, row0, C);
    mm<NK, NP, NPI, NP, false, true>(F, Mb + row0 * kLdc * 2, kLdc, PT, kb + kcol * 2, LD, PK, 0, row0 + 16);
    mm<NK, NP, NPI, NP, true, true>(F, Mb + row0 * 2, kLdc, PT, kb + kcol * 2, LD, PK, row0, C);
#pragma unroll
    for (int n = 0; n < NK; ++n)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            const int i = row0 + acc_row(hf), j = kcol + acc_col(n);
            if (i >= ch.n) continue;
            const int64_t at = ((int64_t)(ch.tok0 + i) * a.Hv + h) * DK + j;
            if (a.part) {
                store2(a.part + at, dq[n][2 * hf], dq[n][2 * hf + 1]);
                store2(a.part + a.T * a.Hv * DK + at, F[n][2 * hf], F[n][2 * hf + 1]);
            } else {
                store2(static_cast<E *>(a.dq) + at, dq[n][2 * hf], dq[n][2 * hf + 1]);
                store2(static_cast<E *>(a.dk_) + at, F[n][2 * hf], F[n][2 * hf + 1]);
            }
        }
}

// ------------------------------------------------------------ shared key heads
// dq and dk of a key head: the sum over its value heads, in their order, rounded once.
template <typename E>
__global__ void __launch_bounds__(kThreads) delta_sum_kernel(const DeltaArgs a) {
    wait_ahead();
    if (a.hdr->bad) return;
    const int share = a.Hv / a.Hk, vec = a.dk / 4;
    const int64_t t0 = a.cu[0], t1 = a.cu[a.N], n = (t1 - t0) * a.Hk * vec;
    for (int64_t i = blockIdx.x * (int64_t)kThreads + threadIdx.x; i < 2 * n; i += (int64_t)gridDim.x * kThreads) {
        const int which = i >= n;
        const int64_t j = (which ? i - n : i) + t0 * a.Hk * vec, head = j / vec;
        const float *p = a.part + (which ? a.T * a.Hv * a.dk : 0) + head * share * a.dk + j % vec * 4;
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int m = 0; m < share; ++m) {
            const float4 x = *reinterpret_cast<const float4 *>(p + (int64_t)m * a.dk);
            s.x += x.x, s.y += x.y, s.z += x.z, s.w += x.w;
        }
        E *o = static_cast<E *>(which ? a.dk_ : a.dq) + j * 4;
        store2(o, s.x, s.y);
        store2(o + 2, s.z, s.w);
    }
}

template <typename E, int DK, int DVS>
cudaError_t back(const DeltaArgs &a, cudaStream_t st) {
    static LaunchFit fit;
    auto kernel = delta_back_kernel<E, DK, DVS>;
    const size_t smem = sizeof(BackSmem<E, DK, DVS>);
    static_assert(sizeof(BackSmem<E, DK, DVS>) <= 232448, "shared memory of one CTA");
    const cudaError_t e = fit.prepare(reinterpret_cast<const void *>(kernel), kThreads, smem, nullptr);
    if (e != cudaSuccess) return e;
    return launch_next(kernel, dim3((unsigned)(a.N * a.Hv * (a.dv / DVS))), kThreads, smem, st, a);
}
template <typename E, int DK, int R>
cudaError_t grads(const DeltaArgs &a, cudaStream_t st) {
    static LaunchFit fit;
    auto kernel = delta_grads_kernel<E, DK, R>;
    const size_t smem = sizeof(GradSmem<E, DK>);
    static_assert(sizeof(GradSmem<E, DK>) <= 232448, "shared memory of one CTA");
    const cudaError_t e = fit.prepare(reinterpret_cast<const void *>(kernel), kThreads, smem, nullptr);
    if (e != cudaSuccess) return e;
    return launch_next<R>(kernel, dim3(a.max_chunks * R, a.Hv), kThreads, smem, st, a);
}
// Two CTAs a cell while every CTA has an SM: a cell's time is its warp-level products' (fp32, 5 chunks of 2 heads of 64 by
// 128: 31.2 -> 26.5 us).
template <typename E, int DK>
cudaError_t grads(const DeltaArgs &a, cudaStream_t st) {
    return (int64_t)a.max_chunks * a.Hv * 2 <= paged_sms() ? grads<E, DK, 2>(a, st) : grads<E, DK, 1>(a, st);
}

}  // namespace

cudaError_t launch_delta_back(const DeltaArgs &a, cudaStream_t st) {
    if (a.dtype == RA_FP32) return a.dk == 64 ? back<float, 64, 32>(a, st) : back<float, 128, 32>(a, st);
    // (slices as narrow as leaves every CTA an SM: 12 sequences of up to 39 tokens, 2 heads of 64, both walks 41.9 -> 38.0 us)
    if ((int64_t)a.N * a.Hv * (a.dv / 32) <= paged_sms())
        return a.dk == 64 ? back<bf16, 64, 32>(a, st) : back<bf16, 128, 32>(a, st);
    return a.dk == 64 ? back<bf16, 64, 64>(a, st) : back<bf16, 128, 64>(a, st);
}
cudaError_t launch_delta_grads(const DeltaArgs &a, cudaStream_t st) {
    if (a.Hv != a.Hk && !a.part) return cudaErrorInvalidValue;  // (several heads would write one place)
    if (a.dtype == RA_FP32) return a.dk == 64 ? grads<float, 64>(a, st) : grads<float, 128>(a, st);
    return a.dk == 64 ? grads<bf16, 64>(a, st) : grads<bf16, 128>(a, st);
}
cudaError_t launch_delta_sum(const DeltaArgs &a, cudaStream_t st) {
    const int64_t n = 2 * a.T * a.Hk * (a.dk / 4);
    const unsigned grid = (unsigned)((n + kThreads - 1) / kThreads < 8192 ? (n + kThreads - 1) / kThreads : 8192);
    return launch_next(a.dtype == RA_FP32 ? delta_sum_kernel<float> : delta_sum_kernel<bf16>, dim3(grid), kThreads, 0, st, a);
}

}  // namespace ra

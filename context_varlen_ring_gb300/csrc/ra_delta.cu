// ra_delta.cu -- the gated delta rule forward: packed sequences chunk by
// chunk, and one token of each sequence against its state.
//
// A head's state S [dk, dv] takes up one token after another:
//   S <- e^g S;  u = beta (v - S^T k);  S <- S + k u^T;  o = scale S^T q.
// Over a chunk of 64 tokens with the state S0 ahead of it, and G the running
// sums of g in the chunk, D_ij = exp(G_i - G_j) for j <= i:
//   A_ij = beta_i D_ij k_i.k_j (j < i),   T = (I + A)^-1
//   r = v - e^G (K S0),   u = T (beta r)
//   o = scale e^G (Q S0) + P u,   P_ij = scale D_ij q_i.k_j (j <= i)
//   S1 = e^(G_63) S0 + K^T (e^(G_63 - G) u)
// T and P need no state: one kernel makes them for all chunks at once.  A
// second one walks each sequence's chunks, a CTA for each head and slice of
// the state's columns (columns never meet), the state in registers: a chain,
// bound by what a chunk takes from its first product to its last (fp32, heads of
// 64: 11,400 cycles with slices of 32 columns).  The one-token form is bound by
// memory, each state read and written once (64 sequences, 32 heads: 45 us, 6.0
// TB/s).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "ra_delta.cuh"
#include "ra_serve.cuh"

namespace ra {
namespace {

using namespace delta;

// ------------------------------------------------------------ plan
// The chunks of all sequences, and the sequences by their number of chunks
// (the longest walk begins first).  One block.
constexpr int kPlanThreads = 1024;
// More sequences stay in their order: a place is a count over all of them, so the order costs with their square (10 us for
// 512, 37 for 1024, 150 for 2048, 600 for 4096).  What it gains depends on where the long ones stand: with one of 8192
// tokens behind short ones (4 heads of 128) 256 sequences take 666 us in order and 770 without, 1024 887 and 1287, 2048
// 1580 and 1988; all of one kind (up to 300 tokens), 256 take 121 and 128, 1024 477 and 447, 2048 987 and 854, 4096 2221
// and 1640.
constexpr int kPlanSort = 2048;

__global__ void __launch_bounds__(kPlanThreads) delta_plan_kernel(const DeltaArgs a) {
    __shared__ int warp_sum[32], carry, bad;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) carry = bad = 0;
    __syncthreads();
    for (int s0 = 0; s0 < a.N; s0 += kPlanThreads) {
        const int s = s0 + tid;
        int c0 = 0, n = 0;
        if (s < a.N) {
            c0 = a.cu[s];
            const int c1 = a.cu[s + 1];
            if (c0 < 0 || c1 < c0 || c1 > a.T)
                bad = 1;
            else
                n = (c1 - c0 + C - 1) / C;
        }
        __syncthreads();
        if (bad) n = 0;
        int sum = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += x;
        }
        if (lane == 31) warp_sum[warp] = sum;
        __syncthreads();
        int at = carry + sum - n;
        for (int i = 0; i < warp; ++i) at += warp_sum[i];
        if (s < a.N) a.first[s] = at;
        __syncthreads();
        if (tid == kPlanThreads - 1) carry = at + n;
        __syncthreads();
    }
    // (boundaries that start above 0 leave the tokens ahead of them alone)
    const int total = min(carry, a.max_chunks);
    if (tid == 0) {
        a.first[a.N] = total;
        a.hdr->chunks = bad ? 0 : total;
        a.hdr->bad = bad;
        if (bad) record_status(a.status, RA_ERR_DEVICE_BOUNDS);
    }
    __syncthreads();
    if (bad) return;
    for (int i = tid; i < total; i += kPlanThreads) {
        int lo = 0, hi = a.N;  // the last sequence that begins at or ahead of chunk i
        while (hi - lo > 1) {
            const int m = (lo + hi) / 2;
            if (a.first[m] <= i)
                lo = m;
            else
                hi = m;
        }
        const int t = a.cu[lo] + (i - a.first[lo]) * C;
        a.chunk[i] = DeltaChunk{t, min(C, a.cu[lo + 1] - t)};
    }
    for (int s = tid; s < a.N; s += kPlanThreads) {
        int rank = s;
        if (a.N <= kPlanSort) {
            const int n = a.first[s + 1] - a.first[s];
            rank = 0;
            for (int i = 0; i < a.N; ++i) {
                const int m = a.first[i + 1] - a.first[i];
                rank += m > n || (m == n && i < s);
            }
        }
        a.order[rank] = s;
    }
}

// ------------------------------------------------------------ T and P
// Floor: what it writes, 16 KB a chunk and head for each of the three parts.  Bound: each chunk is a chain of small steps,
// an SM holds three, and shared memory's port is busy most of the time (its K, Q, A, T and P, all read and written in
// pieces of 16 bytes): 8576 chunks 184 us, 3.5 TB/s.  So half of the warps make A and its inverse, the other half P (with
// two parts 264 us with all of it in four warps, 208 so), what is made takes the place of K and Q, P a part at a time
// (160), and the gates and the diagonal's blocks are read 8 and 16 bytes at a time (160 -> 135).  (I + A)^-1: the 16 x 16 blocks on the diagonal by substitution, a
// lane a column; then blocks of 32 and of 64 from their halves, [T11, 0; -T22 A21 T11, T22], as products of parts.
constexpr int kLocalThreads = 256;
constexpr int kLdy = 40;

template <typename E, int DK>
struct LocalSmem {
    static constexpr int NPI = std::is_same<E, float>::value ? 3 : 1, LD = DK + 8;
    struct Rows {
        bf16 k[NPI][C][LD], q[NPI][C][LD];
    };
    struct Made {
        bf16 P[C][kLdc], A[NP][C][kLdc], T[NP][C][kLdc];
        union {
            alignas(16) float diag[4][16][20];
            bf16 Y[NP][32][kLdy];  // when the diagonal's blocks are inverted
        };
    };
    union {
        Rows in;
        Made made;  // when the products with K and Q are done
    };
    Gates g;
};

template <typename E, int DK>
__global__ void __launch_bounds__(kLocalThreads) delta_local_kernel(const DeltaArgs a) {
    using Smem = LocalSmem<E, DK>;
    constexpr int NPI = Smem::NPI, LD = Smem::LD, PL = C * LD * 2, PT = C * kLdc * 2, PY = 32 * kLdy * 2;
    extern __shared__ __align__(128) uint8_t raw[];
    Smem &sm = *reinterpret_cast<Smem *>(raw);
    const int c = blockIdx.x, h = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    wait_ahead();
    if (c >= a.hdr->chunks) return;
    const DeltaChunk ch = a.chunk[c];
    const int hk = h / (a.Hv / a.Hk);
    const E *k = static_cast<const E *>(a.k) + ch.tok0 * a.k_stride + hk * DK;
    const E *q = static_cast<const E *>(a.q) + ch.tok0 * a.q_stride + hk * DK;
    load_rows<E, DK, kLocalThreads>(&sm.in.k[0][0][0], LD, C * LD, k, a.k_stride, ch.n);
    load_rows<E, DK, kLocalThreads>(&sm.in.q[0][0][0], LD, C * LD, q, a.q_stride, ch.n);
    cp_commit();
    if (warp == 0) {
        float g[2], b[2];
        gates_load(a, ch, h, g, b);
        gates_put(sm.g, g, b);
    }
    cp_wait<0>();
    __syncthreads();
    // rows 16 (warp % 4) .. of K K^T (warps 0 to 3) or Q K^T (4 to 7), up to the diagonal
    const int w = warp & 3, row0 = 16 * w;
    const bool own = warp < 4;
    const uint32_t kb = smem_u32(sm.in.k), row = row0 * LD * 2;
    float x[8][4];
    zero(x);
    mm<8, NPI, NPI, 3, false, false>(x, (own ? kb : smem_u32(sm.in.q)) + row, LD, PL, kb, LD, PL, 0, DK, w + 1);
    __syncthreads();  // (what is made of them takes the place of K and Q)
    float2 Gi[2];
    float f[2];
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
        const int i = row0 + acc_row(hf);
        Gi[hf] = make_float2(sm.g.hi[i], sm.g.lo[i]);
        f[hf] = own ? sm.g.beta[i] : a.scale;
    }
#pragma unroll
    for (int n = 0; n < 8; ++n) {
        const int j = acc_col(n);
        const float2 hi = *reinterpret_cast<const float2 *>(sm.g.hi + j), lo = *reinterpret_cast<const float2 *>(sm.g.lo + j);
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            const int i = row0 + acc_row(hf);
            float y[2] = {0.f, 0.f};
            if (n / 2 <= w) {
                if (j + own <= i) y[0] = f[hf] * gate_exp(Gi[hf], make_float2(hi.x, lo.x)) * x[n][2 * hf];
                if (j + 1 + own <= i) y[1] = f[hf] * gate_exp(Gi[hf], make_float2(hi.y, lo.y)) * x[n][2 * hf + 1];
            }
            if (!own) {
                x[n][2 * hf] = y[0];
                x[n][2 * hf + 1] = y[1];
            } else if (n / 2 <= w) {
                put2<NP>(&sm.made.A[0][i][j], C * kLdc, y[0], y[1]);
                if (n / 2 == w) {
                    *reinterpret_cast<float2 *>(&sm.made.diag[w][i & 15][j & 15]) = make_float2(y[0], y[1]);
                }
            } else {
                put2<NP>(&sm.made.T[0][i][j], C * kLdc, 0.f, 0.f);
            }
        }
    }
    uint16_t *tp = a.tp + ((int64_t)c * a.Hv + h) * 2 * NP * C * C;
    if (!own) {
#pragma unroll
        for (int p = 0; p < NP; ++p) {  // (a part at a time: three CTAs an SM)
#pragma unroll
            for (int n = 0; n < 8; ++n)
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    float *y = x[n] + 2 * hf;
                    const __nv_bfloat162 b = __floats2bfloat162_rn(y[0], y[1]);
                    *reinterpret_cast<__nv_bfloat162 *>(&sm.made.P[row0 + acc_row(hf)][acc_col(n)]) = b;
                    y[0] -= __low2float(b);
                    y[1] -= __high2float(b);
                }
            asm volatile("bar.sync 2, 128;" ::: "memory");
            store_square<1, 128>(tp + (NP + p) * C * C, &sm.made.P[0][0]);
            asm volatile("bar.sync 2, 128;" ::: "memory");
        }
        return;
    }
    auto sync = [] { asm volatile("bar.sync 1, 128;" ::: "memory"); };  // (of the four that go on)
    __syncwarp();
    if (lane < 16) {
        float t[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float s = i == lane ? 1.f : 0.f;
#pragma unroll
            for (int m = 0; m < i; m += 4) {
                const float4 d = *reinterpret_cast<const float4 *>(&sm.made.diag[w][i][m]);
                s -= d.x * t[m];
                if (m + 1 < i) s -= d.y * t[m + 1];
                if (m + 2 < i) s -= d.z * t[m + 2];
                if (m + 3 < i) s -= d.w * t[m + 3];
            }
            t[i] = s;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float s = t[i];
#pragma unroll
            for (int p = 0; p < NP; ++p) {
                const bf16 b = __float2bfloat16_rn(s);
                sm.made.T[p][row0 + i][row0 + lane] = b;
                s -= __bfloat162float(b);
            }
        }
    }
    sync();
    const uint32_t Ab = smem_u32(sm.made.A), Tb = smem_u32(sm.made.T), Yb = smem_u32(sm.made.Y);
    auto tile = [&](uint32_t b, int r, int col) { return b + (r * kLdc + col) * 2; };
    auto put = [&](bf16 *dst, int ld, int plane, const float (&x)[2][4], float sign) {
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf)
                put2<NP>(dst + acc_row(hf) * ld + acc_col(n), plane, sign * x[n][2 * hf], sign * x[n][2 * hf + 1]);
    };
    float y[2][4];
    if (w & 1) {  // rows 16 .. 31 by columns 0 .. 15, and 48 .. by 32 ..
        zero(y);
        mm<2, NP, NP, NP, false, true>(y, tile(Ab, row0, row0 - 16), kLdc, PT, tile(Tb, row0 - 16, row0 - 16), kLdc, PT, 0, 16);
        put(&sm.made.Y[0][(w >> 1) * 16][0], kLdy, 32 * kLdy, y, 1.f);
        __syncwarp();
        zero(y);
        mm<2, NP, NP, NP, false, true>(y, tile(Tb, row0, row0), kLdc, PT, Yb + (w >> 1) * 16 * kLdy * 2, kLdy, PY, 0, 16);
        put(&sm.made.T[0][row0][row0 - 16], kLdc, C * kLdc, y, -1.f);
    }
    sync();
    {  // rows 32 .. 63 by columns 0 .. 31: a block of 16 x 16 each warp
        const int r = (w >> 1) * 16, col = (w & 1) * 16;
        zero(y);
        mm<2, NP, NP, NP, false, true>(y, tile(Ab, 32 + r, 0), kLdc, PT, tile(Tb, 0, col), kLdc, PT, col, 32);
        put(&sm.made.Y[0][r][col], kLdy, 32 * kLdy, y, 1.f);
        sync();
        zero(y);
        mm<2, NP, NP, NP, false, true>(y, tile(Tb, 32 + r, 32), kLdc, PT, Yb + col * 2, kLdy, PY, 0, r + 16);
        put(&sm.made.T[0][32 + r][col], kLdc, C * kLdc, y, -1.f);
    }
    sync();
    store_square<NP, 128>(tp, &sm.made.T[0][0][0]);
}

// ------------------------------------------------------------ the walk
constexpr int kScanThreads = 256;

template <typename E, int DK, int DVS>
struct ScanSmem {
    static constexpr bool F = std::is_same<E, float>::value;
    static constexpr int NPI = F ? 3 : 1, KB = F ? 1 : 2, LD = DK + 8, LV = DVS + 8;
    bf16 k[KB][NPI][C][LD], q[NPI][C][LD];
    bf16 T[NP][C][kLdc], P[NP][C][kLdc];
    bf16 S[NP][DK][LV], R[NP][C][LV], U[NP][C][LV];
    Gates g[2];
};

template <typename E, int DK, int DVS>
__global__ void __launch_bounds__(kScanThreads, 1) delta_scan_kernel(const DeltaArgs a, int keep) {
    using Smem = ScanSmem<E, DK, DVS>;
    constexpr int NPI = Smem::NPI, KB = Smem::KB, LD = Smem::LD, LV = Smem::LV;
    // Slices of 32 or 64 columns: every warp has 16 rows and half of the columns.  Of 16: warps 0 .. 3 have the chain (K S0, T R
    // and, with dk 64, the state), and warps 4 .. 7 the output.
    constexpr bool kRoles = DVS == 16;
    constexpr int MW = DK / 16, MS = kRoles && MW == 4 ? 4 : 8;  // warps along dk, and those with rows of S
    constexpr int NS = DVS / 8 / (MS / MW), NX = kRoles ? 2 : DVS / 16;  // n-tiles of a warp: of S, of rows of the chunk
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
    const int srow = 16 * (warp % MW), scol = warp / MW * 8 * NS;  // this warp's part of S
    const int xrow = 16 * (warp & 3), xcol = kRoles ? 0 : (warp >> 2) * 8 * NX;  // and of the chunk's rows
    const bool chain = !kRoles || warp < 4, state = warp < MS;
    const int64_t slot = a.state || a.state_out ? slot_of(a.slots, a.n_slots, seq, a.status) : -1;
    const int64_t splace = ((slot * a.Hv + h) * DK) * dv + v0;

    float S[NS][4];
#pragma unroll
    for (int n = 0; n < NS; ++n)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            float2 x = make_float2(0.f, 0.f);
            if (a.state && slot >= 0 && state)
                x = *reinterpret_cast<const float2 *>(a.state + splace + (int64_t)(srow + acc_row(hf)) * dv + scol + acc_col(n));
            S[n][2 * hf] = x.x;
            S[n][2 * hf + 1] = x.y;
        }

    auto load_k = [&](int c, int buf) {
        const DeltaChunk ch = a.chunk[c];
        load_rows<E, DK, kScanThreads>(&sm.k[buf][0][0][0], LD, C * LD, static_cast<const E *>(a.k) + ch.tok0 * a.k_stride + hk * DK,
                                       a.k_stride, ch.n);
    };
    auto load_q = [&](int c) {
        const DeltaChunk ch = a.chunk[c];
        load_rows<E, DK, kScanThreads>(&sm.q[0][0][0], LD, C * LD, static_cast<const E *>(a.q) + ch.tok0 * a.q_stride + hk * DK,
                                       a.q_stride, ch.n);
    };
    RowsAhead<DK, kScanThreads> k_ahead, q_ahead;  // (fp32: K and Q of the next chunk)
    auto fetch = [&](int c, bool with_q) {
        const DeltaChunk ch = a.chunk[c];
        k_ahead.fetch(static_cast<const float *>(a.k) + ch.tok0 * a.k_stride + hk * DK, a.k_stride, ch.n);
        if (with_q) q_ahead.fetch(static_cast<const float *>(a.q) + ch.tok0 * a.q_stride + hk * DK, a.q_stride, ch.n);
    };
    auto load_tp = [&](int c, int which) {
        load_square<NP, kScanThreads>(which ? &sm.P[0][0][0] : &sm.T[0][0][0],
                                      a.tp + (((int64_t)c * a.Hv + h) * 2 + which) * NP * C * C);
    };
    const bool want = a.out != nullptr, output = want && (!kRoles || warp >= 4);
    float gg[2], gb[2];
    if (c0 < c1) {
        if (KB == 2) load_k(c0, 0);
        cp_commit();
        if (KB == 2 && want) load_q(c0);
        cp_commit();
        load_tp(c0, 0);
        cp_commit();
        if (want) load_tp(c0, 1);
        cp_commit();
        if (warp == 0) gates_load(a, a.chunk[c0], h, gg, gb);
        if (KB == 1) fetch(c0, want);
    }
    for (int c = c0; c < c1; ++c) {
        const int buf = KB == 2 ? (c - c0) & 1 : 0;
        const DeltaChunk ch = a.chunk[c];
        Gates &g = sm.g[(c - c0) & 1];
        const int64_t cell = (int64_t)c * a.Hv + h;
        if (KB == 1) {
            __syncthreads();  // (the last chunk's products with K)
            k_ahead.put(&sm.k[0][0][0][0], LD, C * LD);
            if (want) q_ahead.put(&sm.q[0][0][0], LD, C * LD);
            if (c + 1 < c1) fetch(c + 1, want);
        }
        if (warp == 0) {
            gates_put(g, gg, gb);
            if (c + 1 < c1) gates_load(a, a.chunk[c + 1], h, gg, gb);
        }
        // the values of this thread's places
        float2 v[NX][2];
#pragma unroll
        for (int n = 0; n < NX; ++n)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const int i = xrow + acc_row(hf);
                v[n][hf] = make_float2(0.f, 0.f);
                if (i < ch.n && chain)
                    v[n][hf] = load2(static_cast<const E *>(a.v) + (ch.tok0 + i) * a.v_stride + h * dv + v0 + xcol + acc_col(n));
            }
        // the state's parts
#pragma unroll
        for (int n = 0; n < NS && state; ++n)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const int i = srow + acc_row(hf), j = scol + acc_col(n);
                put2<NP>(&sm.S[0][i][j], DK * LV, S[n][2 * hf], S[n][2 * hf + 1]);
                if (keep)
                    *reinterpret_cast<float2 *>(a.s0 + (cell * DK + i) * dv + v0 + j) =
                        make_float2(S[n][2 * hf], S[n][2 * hf + 1]);
            }
        cp_wait<2>();  // K and Q
        __syncthreads();
        if (KB == 2 && c + 1 < c1) load_k(c + 1, buf ^ 1);
        cp_commit();
        float x[NX][4], o[NX][4];
        zero(x);
        if (chain)
            mm<NX, NPI, NP, NP, false, true>(x, smem_u32(sm.k[buf]) + xrow * LD * 2, LD, PK, smem_u32(sm.S) + xcol * 2, LV, PS,
                                                 0, DK);
        if (output) {
            zero(o);
            mm<NX, NPI, NP, NP, false, true>(o, smem_u32(sm.q) + xrow * LD * 2, LD, PK, smem_u32(sm.S) + xcol * 2, LV, PS, 0,
                                             DK);
        }
#pragma unroll
        for (int n = 0; n < NX; ++n)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const int i = xrow + acc_row(hf), j = xcol + acc_col(n);
                const float e = g.eG[i], b = g.beta[i];
                const float r0 = v[n][hf].x - e * x[n][2 * hf], r1 = v[n][hf].y - e * x[n][2 * hf + 1];
                if (chain) {
                    put2<NP>(&sm.R[0][i][j], C * LV, b * r0, b * r1);
                    if (keep) *reinterpret_cast<float2 *>(a.r + (cell * C + i) * dv + v0 + j) = make_float2(r0, r1);
                }
                if (output) {
                    o[n][2 * hf] *= e * a.scale;
                    o[n][2 * hf + 1] *= e * a.scale;
                }
            }
        cp_wait<2>();  // T
        __syncthreads();
        if (KB == 2 && want && c + 1 < c1) load_q(c + 1);
        cp_commit();
        zero(x);
        if (chain)
            mm<NX, NP, NP, NP, false, true>(x, smem_u32(sm.T) + xrow * kLdc * 2, kLdc, PT, smem_u32(sm.R) + xcol * 2, LV, PR,
                                                0, xrow + 16);
#pragma unroll
        for (int n = 0; n < NX && chain; ++n)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const int i = xrow + acc_row(hf), j = xcol + acc_col(n);
                if (want) put2<NP>(&sm.U[0][i][j], C * LV, x[n][2 * hf], x[n][2 * hf + 1]);
                if (keep)
                    *reinterpret_cast<float2 *>(a.u + (cell * C + i) * dv + v0 + j) =
                        make_float2(x[n][2 * hf], x[n][2 * hf + 1]);
            }
        cp_wait<2>();  // P
        __syncthreads();
        if (c + 1 < c1) load_tp(c + 1, 0);
        cp_commit();
#pragma unroll
        for (int n = 0; n < NX && chain; ++n)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const int i = xrow + acc_row(hf), j = xcol + acc_col(n);
                put2<NP>(&sm.R[0][i][j], C * LV, g.eL[i] * x[n][2 * hf], g.eL[i] * x[n][2 * hf + 1]);
            }
        if (output) {
            mm<NX, NP, NP, NP, false, true>(o, smem_u32(sm.P) + xrow * kLdc * 2, kLdc, PT, smem_u32(sm.U) + xcol * 2, LV, PR,
                                            0, xrow + 16);
#pragma unroll
            for (int n = 0; n < NX; ++n)
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    const int i = xrow + acc_row(hf);
                    if (i < ch.n)
                        store2(static_cast<E *>(a.out) + ((int64_t)(ch.tok0 + i) * a.Hv + h) * dv + v0 + xcol + acc_col(n),
                               o[n][2 * hf], o[n][2 * hf + 1]);
                }
        }
        __syncthreads();
        if (want && c + 1 < c1) load_tp(c + 1, 1);
        cp_commit();
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) S[n][i] *= g.eC;
        if (state)
            mm<NS, NPI, NP, NP, true, true>(S, smem_u32(sm.k[buf]) + srow * 2, LD, PK, smem_u32(sm.R) + scol * 2, LV, PR, 0, C);
    }
    cp_wait<0>();
    if (a.state_out && slot >= 0 && state) {
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf)
                *reinterpret_cast<float2 *>(a.state_out + splace + (int64_t)(srow + acc_row(hf)) * dv + scol + acc_col(n)) =
                    make_float2(S[n][2 * hf], S[n][2 * hf + 1]);
    }
}

// ------------------------------------------------------------ one token
// Bound: memory, the state read and written once.  A CTA takes 32 columns of
// one head's state (128 bytes a row), a thread four columns of DK / 16 rows,
// all of them loaded before any is used.  S^T k and S^T q are summed together
// and the output is S^T q + (k.q) u, so the rows meet once.
constexpr int kStepThreads = 128;

template <typename E, int DK>
__global__ void __launch_bounds__(kStepThreads) delta_step_kernel(const DeltaStepArgs a) {
    constexpr int ROWS = DK / 16;
    __shared__ float sk[DK], sq[DK], kq[4];
    __shared__ float4 red[2][4][8];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int parts = a.dv / 32, b = blockIdx.x / (a.Hv * parts), h = blockIdx.x / parts % a.Hv, v0 = blockIdx.x % parts * 32;
    const int hk = h / (a.Hv / a.Hk);
    const int64_t slot = slot_of(a.slots, a.n_slots, b, a.status);
    const int rg = tid >> 3, c4 = (tid & 7) * 4;
    E *out = static_cast<E *>(a.out) + ((int64_t)b * a.Hv + h) * a.dv + v0;
    if (slot < 0) {  // a padded batch: no state, no output
        if (tid < 16) store2(out + 2 * tid, 0.f, 0.f);
        return;
    }
    float *S = a.state + ((slot * a.Hv + h) * DK + rg) * a.dv + v0 + c4;
    float4 s[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) s[i] = *reinterpret_cast<const float4 *>(S + (int64_t)i * 16 * a.dv);
    const E *k = static_cast<const E *>(a.k) + b * a.k_stride + hk * DK, *q = static_cast<const E *>(a.q) + b * a.q_stride + hk * DK;
    float dot = 0.f;
    for (int i = tid; i < DK; i += kStepThreads) {
        sk[i] = (float)k[i];
        sq[i] = (float)q[i];
        dot += sk[i] * sq[i];
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
    if (lane == 0) kq[warp] = dot;
    const E *vp = static_cast<const E *>(a.v) + b * a.v_stride + h * a.dv + v0 + c4;
    const float2 va = load2(vp), vb = load2(vp + 2);
    const float decay = expf(__ldg(a.g + (int64_t)b * a.Hv + h)), beta = __ldg(a.beta + (int64_t)b * a.Hv + h);
    __syncthreads();
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const float kk = sk[rg + 16 * i], qq = sq[rg + 16 * i];
        s[i].x *= decay, s[i].y *= decay, s[i].z *= decay, s[i].w *= decay;
        x.x += s[i].x * kk, x.y += s[i].y * kk, x.z += s[i].z * kk, x.w += s[i].w * kk;
        y.x += s[i].x * qq, y.y += s[i].y * qq, y.z += s[i].z * qq, y.w += s[i].w * qq;
    }
#pragma unroll
    for (int o = 8; o <= 16; o <<= 1) {
        x.x += __shfl_xor_sync(0xffffffffu, x.x, o), x.y += __shfl_xor_sync(0xffffffffu, x.y, o);
        x.z += __shfl_xor_sync(0xffffffffu, x.z, o), x.w += __shfl_xor_sync(0xffffffffu, x.w, o);
        y.x += __shfl_xor_sync(0xffffffffu, y.x, o), y.y += __shfl_xor_sync(0xffffffffu, y.y, o);
        y.z += __shfl_xor_sync(0xffffffffu, y.z, o), y.w += __shfl_xor_sync(0xffffffffu, y.w, o);
    }
    if (lane < 8) {
        red[0][warp][lane] = x;
        red[1][warp][lane] = y;
    }
    __syncthreads();
    x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
    dot = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        const float4 p = red[0][w][tid & 7], r = red[1][w][tid & 7];
        x.x += p.x, x.y += p.y, x.z += p.z, x.w += p.w;
        y.x += r.x, y.y += r.y, y.z += r.z, y.w += r.w;
        dot += kq[w];
    }
    const float4 u = make_float4(beta * (va.x - x.x), beta * (va.y - x.y), beta * (vb.x - x.z), beta * (vb.y - x.w));
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const float kk = sk[rg + 16 * i];
        s[i].x += kk * u.x, s[i].y += kk * u.y, s[i].z += kk * u.z, s[i].w += kk * u.w;
        *reinterpret_cast<float4 *>(S + (int64_t)i * 16 * a.dv) = s[i];
    }
    if (tid < 8) {
        store2(out + c4, a.scale * (y.x + dot * u.x), a.scale * (y.y + dot * u.y));
        store2(out + c4 + 2, a.scale * (y.z + dot * u.z), a.scale * (y.w + dot * u.w));
    }
}

template <typename E, int DK>
cudaError_t local(const DeltaArgs &a, cudaStream_t st) {
    static LaunchFit fit;
    auto kernel = delta_local_kernel<E, DK>;
    const size_t smem = sizeof(LocalSmem<E, DK>);
    const cudaError_t e = fit.prepare(reinterpret_cast<const void *>(kernel), kLocalThreads, smem, nullptr);
    if (e != cudaSuccess) return e;
    return launch_next(kernel, dim3(a.max_chunks, a.Hv), kLocalThreads, smem, st, a);
}
template <typename E, int DK, int DVS>
cudaError_t scan(const DeltaArgs &a, int keep, cudaStream_t st) {
    static LaunchFit fit;
    auto kernel = delta_scan_kernel<E, DK, DVS>;
    const size_t smem = sizeof(ScanSmem<E, DK, DVS>);
    static_assert(sizeof(ScanSmem<E, DK, DVS>) <= 232448, "shared memory of one CTA");
    const cudaError_t e = fit.prepare(reinterpret_cast<const void *>(kernel), kScanThreads, smem, nullptr);
    if (e != cudaSuccess) return e;
    return launch_next(kernel, dim3((unsigned)(a.N * a.Hv * (a.dv / DVS))), kScanThreads, smem, st, a, keep);
}

}  // namespace

cudaError_t launch_delta_plan(const DeltaArgs &a, cudaStream_t st) {
    delta_plan_kernel<<<1, kPlanThreads, 0, st>>>(a);
    return cudaGetLastError();
}
cudaError_t launch_delta_local(const DeltaArgs &a, cudaStream_t st) {
    if (a.dtype == RA_FP32) return a.dk == 64 ? local<float, 64>(a, st) : local<float, 128>(a, st);
    return a.dk == 64 ? local<bf16, 64>(a, st) : local<bf16, 128>(a, st);
}
// Slices of the state's columns: a step of the chain is bound by its warp-level products (fp32, dk 64, 32 columns: 5700 of
// 11,400 cycles), so they are as narrow as leaves every CTA an SM (fp32, 5 sequences of up to 292 tokens, 4 heads of 64:
// slices of 32 columns 35.0 us, of 16 28.4; bf16, a sequence of 1408 tokens, one head of 64 by 128: of 64 the call takes
// 161, of 32 113).  With more CTAs than SMs, narrow slices only read K and Q more often.
cudaError_t launch_delta_scan(const DeltaArgs &a, int keep, cudaStream_t st) {
    const int64_t heads = (int64_t)a.N * a.Hv;
    if (a.dtype == RA_FP32) {
        if (heads * (a.dv / 16) <= paged_sms())
            return a.dk == 64 ? scan<float, 64, 16>(a, keep, st) : scan<float, 128, 16>(a, keep, st);
        return a.dk == 64 ? scan<float, 64, 32>(a, keep, st) : scan<float, 128, 32>(a, keep, st);
    }
    const bool few = heads * (a.dv / 32) <= paged_sms();
    if (few) return a.dk == 64 ? scan<bf16, 64, 32>(a, keep, st) : scan<bf16, 128, 32>(a, keep, st);
    return a.dk == 64 ? scan<bf16, 64, 64>(a, keep, st) : scan<bf16, 128, 64>(a, keep, st);
}
cudaError_t launch_delta_step(const DeltaStepArgs &a, cudaStream_t st) {
    const unsigned grid = (unsigned)((int64_t)a.B * a.Hv * (a.dv / 32));
    if (a.dtype == RA_FP32) {
        if (a.dk == 64)
            delta_step_kernel<float, 64><<<grid, kStepThreads, 0, st>>>(a);
        else
            delta_step_kernel<float, 128><<<grid, kStepThreads, 0, st>>>(a);
    } else if (a.dk == 64) {
        delta_step_kernel<bf16, 64><<<grid, kStepThreads, 0, st>>>(a);
    } else {
        delta_step_kernel<bf16, 128><<<grid, kStepThreads, 0, st>>>(a);
    }
    return cudaGetLastError();
}

}  // namespace ra

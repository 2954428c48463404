// ra_delta.cuh -- what the gated delta rule's kernels share: products of tiles
// held as bf16 parts, a chunk's gates, and the loads of its rows.
//
// Arithmetic.  The states, their gradients and the gates' gradients are fp32
// results, so the products' operands have to carry more than bf16's 8 bits: an
// operand that is not bf16 itself is held as the sum of three bf16 parts (24
// bits), and a product adds the parts' products up to the third order, in fp32.
// q, k, v and dout of a bf16 call are one part, exactly.  (A bf16 forward from
// two parts, 16 bits, is faster but up to 5e-6 of the largest result off beside
// its own rounding, and 1.4e-4 of the norm from the rounded exact result; of
// three 5e-8 and 2.9e-5, as plain fp32 arithmetic is.)
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "ra_delta.h"
#include "ra_dev.cuh"

namespace ra {
namespace delta {

using namespace dev;
using bf16 = __nv_bfloat16;
constexpr int C = kDeltaChunk, NP = kDeltaParts;
constexpr int kLdc = C + 8;  // pitch of a [64][64] tile: rows of 9 x 16 bytes, so that eight rows meet eight bank groups

__device__ __forceinline__ void cp16z(uint32_t dst, const void *src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
template <bool TRANS>
__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t (&r)[4]) {
    if (TRANS)
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                     : "r"(a)
                     : "memory");
    else
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                     : "r"(a)
                     : "memory");
}
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// acc[16 x 8 NT] += A[16 x K] B[K x 8 NT] over K = k0 .. k1 - 1 (multiples of
// 16), operands of PA and PB parts, products of parts i, j with i + j < NP.
// a, b: shared addresses of A's and B's first element; lda, ldb: pitches in
// elements; pa, pb: bytes between parts.  TA: A is stored [K][M]; BKN: B is
// stored [K][N], else [N][K].  Every 16 of K are summed by themselves and
// added to acc in fp32, because the tensor cores cut what they add to an
// accumulator, always towards 0 (fp32 gradients off by 1.5e-6 of their norm
// without, 1.6e-7 with).
template <int NT, int PA, int PB, int NP, bool TA, bool BKN>
__device__ __forceinline__ void mm(float (&acc)[NT][4], uint32_t a, int lda, int pa, uint32_t b, int ldb, int pb, int k0,
                                   int k1, int pairs = NT / 2) {
    const int l = threadIdx.x & 31, r = l & 7, s = (l >> 3) & 1, h = l >> 4;
    a += 2 * (TA ? (h * 8 + r) * lda + s * 8 : (s * 8 + r) * lda + h * 8);
    b += 2 * (BKN ? (s * 8 + r) * ldb + h * 8 : (h * 8 + r) * ldb + s * 8);
    const int as = TA ? 2 * lda : 2, bs = BKN ? 2 * ldb : 2, bn = BKN ? 32 : 32 * ldb;
#pragma unroll 2
    for (int k = k0; k < k1; k += 16) {
        uint32_t fa[PA][4];
#pragma unroll
        for (int i = 0; i < PA; ++i) ldsm4<TA>(a + i * pa + k * as, fa[i]);
#pragma unroll
        for (int n = 0; n < NT / 2; ++n) {
            if (n >= pairs) break;
            uint32_t fb[PB][4];
#pragma unroll
            for (int j = 0; j < PB; ++j) ldsm4<BKN>(b + j * pb + k * bs + n * bn, fb[j]);
            float own[2][4] = {};
            // (the small products first)
#pragma unroll
            for (int o = NP - 1; o >= 0; --o)
#pragma unroll
                for (int i = 0; i < PA; ++i) {
                    const int j = o - i;
                    if (j < 0 || j >= PB) continue;
                    mma(own[0], fa[i], fb[j][0], fb[j][1]);
                    mma(own[1], fa[i], fb[j][2], fb[j][3]);
                }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                acc[2 * n][i] += own[0][i];
                acc[2 * n + 1][i] += own[1][i];
            }
        }
    }
}
template <int NT>
__device__ __forceinline__ void zero(float (&acc)[NT][4]) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[n][i] = 0.f;
}

// Two neighbouring elements into NP bf16 parts, `plane` elements apart.
template <int NP>
__device__ __forceinline__ void put2(bf16 *p, int plane, float x, float y) {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
        *reinterpret_cast<__nv_bfloat162 *>(p + i * plane) = h;
        x -= __low2float(h);
        y -= __high2float(h);
    }
}
template <int NP>
__device__ __forceinline__ float2 get2(const bf16 *p, int plane) {
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = NP - 1; i >= 0; --i) {
        const float2 x = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(p + i * plane));
        s.x += x.x;
        s.y += x.y;
    }
    return s;
}
// Row and first column of an accumulator's pair: acc[n][2 half], acc[n][2 half + 1].
__device__ __forceinline__ int acc_row(int half) { return ((threadIdx.x & 31) >> 2) + 8 * half; }
__device__ __forceinline__ int acc_col(int n) { return n * 8 + 2 * (threadIdx.x & 3); }

template <typename E>
__device__ __forceinline__ float2 load2(const E *p) {
    if (std::is_same<E, float>::value) return *reinterpret_cast<const float2 *>(p);
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(p));
}
template <typename E>
__device__ __forceinline__ void store2(E *p, float x, float y) {
    if (std::is_same<E, float>::value)
        *reinterpret_cast<float2 *>(p) = make_float2(x, y);
    else
        *reinterpret_cast<__nv_bfloat162 *>(p) = __floats2bfloat162_rn(x, y);
}

// Rows 0 .. n - 1 of [64][W] elements, `stride` apart, into parts of pitch ld
// (rows behind them zero).  bf16: asynchronous copies, not committed.
template <typename E, int W, int THREADS>
__device__ __forceinline__ void load_rows(bf16 *dst, int ld, int plane, const E *src, int64_t stride, int n) {
    if (std::is_same<E, float>::value) {
        for (int i = threadIdx.x; i < C * (W / 4); i += THREADS) {
            const int row = i / (W / 4), c = i % (W / 4) * 4;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (row < n) x = *reinterpret_cast<const float4 *>(src + row * stride + c);
            put2<3>(dst + row * ld + c, plane, x.x, x.y);
            put2<3>(dst + row * ld + c + 2, plane, x.z, x.w);
        }
    } else {
        for (int i = threadIdx.x; i < C * (W / 8); i += THREADS) {
            const int row = i / (W / 8), c = i % (W / 8) * 8;
            cp16z(smem_u32(dst + row * ld + c), src + (row < n ? row * stride : 0) + c, row < n);
        }
    }
}
// fp32 rows [64][W] by way of registers, so that they can be under way while the tile is in use.
template <int W, int THREADS>
struct RowsAhead {
    float4 x[C * (W / 4) / THREADS];
    __device__ __forceinline__ void fetch(const float *src, int64_t stride, int n) {
#pragma unroll
        for (int e = 0; e < C * (W / 4) / THREADS; ++e) {
            const int i = threadIdx.x + e * THREADS, row = i / (W / 4), c = i % (W / 4) * 4;
            x[e] = row < n ? *reinterpret_cast<const float4 *>(src + row * stride + c) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
    }
    __device__ __forceinline__ void put(bf16 *dst, int ld, int plane) const {
#pragma unroll
        for (int e = 0; e < C * (W / 4) / THREADS; ++e) {
            const int i = threadIdx.x + e * THREADS, row = i / (W / 4), c = i % (W / 4) * 4;
            put2<3>(dst + row * ld + c, plane, x[e].x, x[e].y);
            put2<3>(dst + row * ld + c + 2, plane, x[e].z, x[e].w);
        }
    }
};
// T and P lie in the workspace as tiles that a bulk copy can take to shared memory: a part after another, rows of 128
// bytes whose 16-byte pieces are exchanged by the row's low bits (the 128-byte swizzle of the tensor cores' operands).
__device__ __forceinline__ int swizzled(int row, int piece) { return row * C + ((piece ^ (row & 7)) << 3); }
// Such a tile into parts of pitch kLdc; not committed.
template <int NP, int THREADS>
__device__ __forceinline__ void load_square(bf16 *dst, const uint16_t *src) {
    for (int i = threadIdx.x; i < NP * C * 8; i += THREADS) {
        const int row = i >> 3, c = i & 7;  // (parts one behind another on both sides: whole groups of 8 rows)
        cp16z(smem_u32(dst + row * kLdc + c * 8), src + swizzled(row, c), true);
    }
}
// And back, from parts of pitch kLdc, by a group of THREADS threads.
template <int NP, int THREADS>
__device__ __forceinline__ void store_square(uint16_t *dst, const bf16 *src) {
    for (int i = threadIdx.x % THREADS; i < NP * C * 8; i += THREADS) {
        const int row = i >> 3, c = i & 7;
        *reinterpret_cast<uint4 *>(dst + swizzled(row, c)) = *reinterpret_cast<const uint4 *>(src + row * kLdc + c * 8);
    }
}
// A chunk's gates.  G_i is the sum of its first i + 1 log decays; kept in base 2
// and as the sum of two floats, because the products use exp(G_i - G_j), whose
// exponent would otherwise lose the bits that a strong decay ahead of both pushes
// out.  Decays below -1e4 are e^-1e4 = 0 all the same, and keep the sums finite.
struct alignas(16) Gates {
    float hi[C], lo[C];
    float beta[C];
    float eG[C];     // exp(G_i): the state ahead of the chunk as token i sees it
    float eL[C];     // exp(G_63 - G_i): what token i writes as the chunk's end sees it
    float eC;        // exp(G_63)
};
__device__ __forceinline__ float2 two_sum(float2 a, float2 b) {
    const float s = a.x + b.x, t = s - a.x;
    const float e = (a.x - (s - t)) + (b.x - t) + (a.y + b.y);
    const float h = s + e;
    return make_float2(h, e - (h - s));
}
__device__ __forceinline__ float gate_exp(float2 a, float2 b) { return ex2_approx((a.x - b.x) + (a.y - b.y)); }
// g log2(e), log2(e) = 1.44269502 + 1.92596e-8.
__device__ __forceinline__ float2 in_base_2(float g) {
    const float p = g * 1.44269502f;
    return make_float2(p, fmaf(g, 1.44269502f, -p) + g * 1.92596299e-8f);
}
// The exponential of the gates between tokens j < i (1 at j = i).
__device__ __forceinline__ float decay(const Gates &s, int i, int j) {
    return gate_exp(make_float2(s.hi[i], s.lo[i]), make_float2(s.hi[j], s.lo[j]));
}
// Lane l's log decays and betas of tokens 2 l and 2 l + 1 (0 behind the chunk's n).
__device__ __forceinline__ void gates_load(const DeltaArgs &a, const DeltaChunk &ch, int h, float (&g)[2], float (&b)[2]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int t = 2 * lane + i;
        const int64_t at = (int64_t)(ch.tok0 + t) * a.Hv + h;
        g[i] = t < ch.n ? __ldg(a.g + at) : 0.f;
        b[i] = t < ch.n ? __ldg(a.beta + at) : 0.f;
        if (g[i] < -1e4f) g[i] = -1e4f;
    }
}
// One warp.
__device__ __forceinline__ void gates_put(Gates &s, const float (&g)[2], const float (&b)[2]) {
    const int lane = threadIdx.x & 31;
    const float2 first = in_base_2(g[0]);
    float2 sum = two_sum(first, in_base_2(g[1]));
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const float2 x = make_float2(__shfl_up_sync(0xffffffffu, sum.x, o), __shfl_up_sync(0xffffffffu, sum.y, o));
        if (lane >= o) sum = two_sum(x, sum);
    }
    float2 before = make_float2(__shfl_up_sync(0xffffffffu, sum.x, 1), __shfl_up_sync(0xffffffffu, sum.y, 1));
    if (lane == 0) before = make_float2(0.f, 0.f);
    const float2 last = make_float2(__shfl_sync(0xffffffffu, sum.x, 31), __shfl_sync(0xffffffffu, sum.y, 31));
    const float2 none = make_float2(0.f, 0.f), at[2] = {two_sum(before, first), sum};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int t = 2 * lane + i;
        s.hi[t] = at[i].x;
        s.lo[t] = at[i].y;
        s.beta[t] = b[i];
        s.eG[t] = gate_exp(at[i], none);
        s.eL[t] = gate_exp(last, at[i]);
    }
    if (lane == 0) s.eC = gate_exp(last, none);
}

// The thread of a converged warp that issues products; the same one commits them (tc_commit_w).
__device__ __forceinline__ bool elected() {
    uint32_t e;
    asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\tselp.u32 %0, 1, 0, e;\n\t}\n" : "=r"(e));
    return e != 0;
}

// 16 columns at each of two places, one wait; 32.
__device__ __forceinline__ void tmem_ld16x2(uint32_t a0, uint32_t a1, uint32_t (&x)[16], uint32_t (&y)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%32];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%33];\n\t"
        "tcgen05.wait::ld.sync.aligned;\n"
        : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]), "=r"(x[4]), "=r"(x[5]), "=r"(x[6]), "=r"(x[7]), "=r"(x[8]), "=r"(x[9]), "=r"(x[10]), "=r"(x[11]), "=r"(x[12]), "=r"(x[13]), "=r"(x[14]), "=r"(x[15]),
          "=r"(y[0]), "=r"(y[1]), "=r"(y[2]), "=r"(y[3]), "=r"(y[4]), "=r"(y[5]), "=r"(y[6]), "=r"(y[7]), "=r"(y[8]), "=r"(y[9]), "=r"(y[10]), "=r"(y[11]), "=r"(y[12]), "=r"(y[13]), "=r"(y[14]), "=r"(y[15])
        : "r"(a0), "r"(a1)
        : "memory");
}
__device__ __forceinline__ void tmem_ld32x2(uint32_t a0, uint32_t a1, uint32_t (&x)[32], uint32_t (&y)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%64];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%65];\n\t"
        "tcgen05.wait::ld.sync.aligned;\n"
        : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]), "=r"(x[4]), "=r"(x[5]), "=r"(x[6]), "=r"(x[7]), "=r"(x[8]), "=r"(x[9]), "=r"(x[10]), "=r"(x[11]), "=r"(x[12]), "=r"(x[13]), "=r"(x[14]), "=r"(x[15]), "=r"(x[16]), "=r"(x[17]), "=r"(x[18]), "=r"(x[19]), "=r"(x[20]), "=r"(x[21]), "=r"(x[22]), "=r"(x[23]), "=r"(x[24]), "=r"(x[25]), "=r"(x[26]), "=r"(x[27]), "=r"(x[28]), "=r"(x[29]), "=r"(x[30]), "=r"(x[31]),
          "=r"(y[0]), "=r"(y[1]), "=r"(y[2]), "=r"(y[3]), "=r"(y[4]), "=r"(y[5]), "=r"(y[6]), "=r"(y[7]), "=r"(y[8]), "=r"(y[9]), "=r"(y[10]), "=r"(y[11]), "=r"(y[12]), "=r"(y[13]), "=r"(y[14]), "=r"(y[15]), "=r"(y[16]), "=r"(y[17]), "=r"(y[18]), "=r"(y[19]), "=r"(y[20]), "=r"(y[21]), "=r"(y[22]), "=r"(y[23]), "=r"(y[24]), "=r"(y[25]), "=r"(y[26]), "=r"(y[27]), "=r"(y[28]), "=r"(y[29]), "=r"(y[30]), "=r"(y[31])
        : "r"(a0), "r"(a1)
        : "memory");
}

// The state's place of a sequence in the pool; -1: it has none (a negative slot), or one outside the pool (recorded).
__device__ __forceinline__ int64_t slot_of(const int32_t *slots, int64_t n_slots, int seq, int *status) {
    const int64_t s = slots ? __ldg(slots + seq) : seq;
    if (s >= 0 && s < n_slots) return s;
    if (s >= n_slots) record_status(status, RA_ERR_DEVICE_BOUNDS);
    return -1;
}

// The kernels of a call but the first are launched as programmatic successors: their blocks are set up while the
// kernel ahead ends, and wait for it before they read what it wrote.
__device__ __forceinline__ void wait_ahead() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
template <int CLUSTER = 1, typename... P, typename... A>
cudaError_t launch_next(void (*kernel)(P...), dim3 grid, unsigned block, size_t smem, cudaStream_t st, const A &...args) {
    cudaLaunchAttribute at[2]{};
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = CLUSTER;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t c{};
    c.gridDim = grid;
    c.blockDim = dim3(block);
    c.dynamicSmemBytes = smem;
    c.stream = st;
    c.attrs = at;
    c.numAttrs = CLUSTER > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&c, kernel, args...);
}

}  // namespace delta
}  // namespace ra

// ra_paged.cu -- attention over a paged cache with shared prefixes: the plan
// (who computes what), the SIMT kernel for fp32 and for the shapes that the
// tensor-core kernels do not take, and the kernel that joins the partials.
//
// Mathematics: out = sum_j p_j v_j / sum_j p_j with p_j = 2^(s_j - m), s_j the
// scaled score in base 2 and m the running maximum, over two key sets: the
// prefix of the token's group and its sequence's own keys.  Both sets, and
// the pieces that one set is split into, give partials (m, sum p, sum p v)
// that add after scaling by 2^(m - M).
//
// Split: every (segment, tile of query rows, KV head) is a unit of key tiles.
// All units' tiles form one line, cut into equal runs of tiles, one a CTA, so
// the work is even whatever the lengths, and one long sequence fills the GPU
// as a full batch does.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "ra_dev.cuh"
#include "ra_kernels.h"
#include "ra_paged.cuh"

namespace ra {
namespace {

using namespace dev;

// ------------------------------------------------------------------ plan
constexpr int kPlanThreads = 512;
constexpr int kPlanHeld = 2048;  // segments whose places are searched in shared memory

struct UW {
    long long u, w;  // partial rows, key tiles
};

// Exclusive scan over the block; `total` is the block's sum.
__device__ __forceinline__ UW block_scan(UW v, UW *warp_sum, UW &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    UW x = v;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, x.u, s);
        const long long w = __shfl_up_sync(0xffffffffu, x.w, s);
        if (lane >= s) {
            x.u += u;
            x.w += w;
        }
    }
    if (lane == 31) warp_sum[warp] = x;
    __syncthreads();
    UW before{0, 0};
    total = UW{0, 0};
    for (int i = 0; i < kPlanThreads / 32; ++i) {
        if (i < warp) {
            before.u += warp_sum[i].u;
            before.w += warp_sum[i].w;
        }
        total.u += warp_sum[i].u;
        total.w += warp_sum[i].w;
    }
    __syncthreads();
    return UW{before.u + x.u - v.u, before.w + x.w - v.w};
}

// A block per family: checks its segment arrays, and writes its segments with
// the tiles and partial rows ahead of each, the tiles a CTA, and the segment
// in which each CTA's run begins.
__global__ void __launch_bounds__(kPlanThreads) paged_plan_kernel(const __grid_constant__ PagedArgs a) {
    __shared__ UW warp_sum[kPlanThreads / 32];
    __shared__ long long ahead[kPlanHeld];
    const int fi = blockIdx.x;
    const PagedFamily &f = a.f[fi];
    pdl_launch();
    int bad = 0;
    UW base{0, 0};
    for (int s0 = 0; s0 < f.S; s0 += kPlanThreads) {
        const int s = s0 + threadIdx.x;
        UW v{0, 0};
        PagedSeg g{};
        if (s < f.S) {
            bad |= !paged_record(a, f, fi, s, g);
            v.u = paged_rows(a, f, g);
            v.w = paged_tiles(a, f, g);
        }
        UW total;
        const UW at = block_scan(v, warp_sum, total);
        if (s < f.S) {
            g.W0 = base.w + at.w;
            g.R0 = base.u + at.u;
            f.seg[s] = g;
            if (s < kPlanHeld) ahead[s] = g.W0;
        }
        base.u += total.u;
        base.w += total.w;
    }
    bad = __syncthreads_or(bad);
    const long long W = bad ? 0 : base.w, per = paged_per(f, W);
    if (threadIdx.x == 0) {
        if (bad) record_status(a.status, RA_ERR_DEVICE_BOUNDS);
        f.hdr->W = W;
        f.hdr->per = per;
        f.hdr->err = bad;
    }
    // CTA c begins at place c * per: in the last segment that begins there or earlier and has tiles behind it
    for (int c = threadIdx.x; c < f.n && c * per < W; c += kPlanThreads) {
        int lo = 0, hi = f.S - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if ((mid < kPlanHeld ? ahead[mid] : f.seg[mid].W0) <= c * per)
                lo = mid;
            else
                hi = mid - 1;
        }
        f.start[c] = lo;  // (segments without tiles share their place with the one behind them: the last is it)
    }
}

// ------------------------------------------------------------------ SIMT
constexpr int kKT = 64;

template <typename T>
__device__ __forceinline__ float4 load4(const T *p) {
    if constexpr (sizeof(T) == 4) {
        return *reinterpret_cast<const float4 *>(p);
    } else {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        const float2 x = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&v.x));
        const float2 y = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&v.y));
        return make_float4(x.x, x.y, y.x, y.y);
    }
}

template <int NV, int RPW, int WARPS>
constexpr size_t simt_smem() {
    return sizeof(float) * ((size_t)kKT * (32 * NV + 4) + (size_t)kKT * 32 * NV + (size_t)RPW * WARPS * 32 * NV +
                            (size_t)RPW * WARPS * kKT);
}

// fp32 arithmetic throughout.  A warp owns RPW query rows: a lane scores keys
// lane and lane + 32 for all of them (K rows padded by one vector, so the
// 16-byte reads of neighbouring keys spread over the banks; Q is broadcast),
// then owns columns lane + 32 e of the products.  FMAs per shared-memory
// wavefront: RPW * 8 / (8 + RPW) in the scores, so 8 rows a warp keep the FMA
// pipe the limit; 4 rows a warp serve the few rows of single-token steps.
template <typename T, int NV, int RPW, int WARPS>
__global__ void __launch_bounds__(WARPS * 32) paged_simt_kernel(const __grid_constant__ PagedArgs a, int fi,
                                                                int late) {
    constexpr int D = 32 * NV, RT = RPW * WARPS, KS = D + 4;
    extern __shared__ float4 smem4[];
    float *Ks = reinterpret_cast<float *>(smem4), *Vs = Ks + kKT * KS, *Qs = Vs + kKT * D, *Ps = Qs + RT * D;
    const PagedFamily &f = a.f[fi];
    if (!late) pdl_wait();
    pdl_launch();
    const int cta = blockIdx.x;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    __shared__ PlanShared plan;
    PagedWalk walk = paged_begin<WARPS * 32>(a, f, fi, plan);
    for (PagedUnit u; paged_unit(a, f, fi, walk, u);) {
        const PagedUnit &g = u;
        const int s = u.s;
        const int R = g.n * a.G, r0 = u.r0;
        __syncthreads();  // the last unit's readers are done with Q
        for (int i = threadIdx.x; i < RT * (D / 4); i += WARPS * 32) {
            const int r = i / (D / 4), c = i % (D / 4) * 4, row = r0 + r;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (row < R) {
                const int t = paged_token(a, row);
                v = load4(static_cast<const T *>(a.q) + (int64_t)(g.tok0 + t) * a.q_stride +
                          (int64_t)(u.h * a.G + row - t * a.G) * D + c);
                v.x *= a.scale_log2;
                v.y *= a.scale_log2;
                v.z *= a.scale_log2;
                v.w *= a.scale_log2;
            }
            *reinterpret_cast<float4 *>(Qs + r * D + c) = v;
        }
        float m[RPW], l[RPW], acc[RPW][NV];
        int limit[RPW];
#pragma unroll
        for (int r = 0; r < RPW; ++r) {
            m[r] = -INFINITY;
            l[r] = 0.f;
#pragma unroll
            for (int e = 0; e < NV; ++e) acc[r][e] = 0.f;
            limit[r] = paged_limit(a, g, fi, r0 + warp * RPW + r);
        }
        for (int tile = u.t0; tile < u.t1; ++tile) {
            const int k0 = tile * kKT;
            __syncthreads();
            // a batch of loads is on its way before the first of it is stored
            constexpr int kEach = kKT * (D / 4) / (WARPS * 32), kBatch = kEach % 8 == 0 ? 8 : kEach % 4 == 0 ? 4 : 2;
            for (int i0 = threadIdx.x; i0 < kKT * (D / 4); i0 += kBatch * WARPS * 32) {
                int64_t off[kBatch];
                float4 kv[kBatch], vv[kBatch];
#pragma unroll
                for (int n = 0; n < kBatch; ++n) off[n] = paged_row(a, f, s, g.len, k0 + (i0 + n * WARPS * 32) / (D / 4));
#pragma unroll
                for (int n = 0; n < kBatch; ++n) {
                    const int c = (i0 + n * WARPS * 32) % (D / 4) * 4;
                    kv[n] = vv[n] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (off[n] >= 0) {
                        kv[n] = load4(static_cast<const T *>(a.k) + off[n] + u.h * a.head_stride + c);
                        vv[n] = load4(static_cast<const T *>(a.v) + off[n] + u.h * a.head_stride + c);
                    }
                }
#pragma unroll
                for (int n = 0; n < kBatch; ++n) {
                    const int i = i0 + n * WARPS * 32, j = i / (D / 4), c = i % (D / 4) * 4;
                    *reinterpret_cast<float4 *>(Ks + j * KS + c) = kv[n];
                    *reinterpret_cast<float4 *>(Vs + j * D + c) = vv[n];
                }
            }
            __syncthreads();
            float s0[RPW], s1[RPW];
#pragma unroll
            for (int r = 0; r < RPW; ++r) s0[r] = s1[r] = 0.f;
            const float *qw = Qs + warp * RPW * D;
#pragma unroll 4
            for (int c = 0; c < D; c += 4) {
                const float4 ka = *reinterpret_cast<const float4 *>(Ks + lane * KS + c);
                const float4 kb = *reinterpret_cast<const float4 *>(Ks + (lane + 32) * KS + c);
#pragma unroll
                for (int r = 0; r < RPW; ++r) {
                    const float4 qv = *reinterpret_cast<const float4 *>(qw + r * D + c);
                    s0[r] = fmaf(qv.x, ka.x, fmaf(qv.y, ka.y, fmaf(qv.z, ka.z, fmaf(qv.w, ka.w, s0[r]))));
                    s1[r] = fmaf(qv.x, kb.x, fmaf(qv.y, kb.y, fmaf(qv.z, kb.z, fmaf(qv.w, kb.w, s1[r]))));
                }
            }
            float *pw = Ps + warp * RPW * kKT;
#pragma unroll
            for (int r = 0; r < RPW; ++r) {
                const float xa = k0 + lane < limit[r] ? s0[r] : -INFINITY;
                const float xb = k0 + lane + 32 < limit[r] ? s1[r] : -INFINITY;
                float mx = fmaxf(xa, xb);
#pragma unroll
                for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                const float mn = fmaxf(m[r], mx), use = mn == -INFINITY ? 0.f : mn;
                const float pa = exp2f(xa - use), pb = exp2f(xb - use), alpha = exp2f(m[r] - use);
                l[r] = l[r] * alpha + pa + pb;  // a lane's own keys; joined at the end
                m[r] = mn;
#pragma unroll
                for (int e = 0; e < NV; ++e) acc[r][e] *= alpha;
                pw[r * kKT + lane] = pa;
                pw[r * kKT + lane + 32] = pb;
            }
            __syncwarp();
#pragma unroll 2
            for (int j = 0; j < kKT; j += 4) {
                float v0[NV], v1[NV], v2[NV], v3[NV];
#pragma unroll
                for (int e = 0; e < NV; ++e) {
                    v0[e] = Vs[j * D + lane + 32 * e];
                    v1[e] = Vs[(j + 1) * D + lane + 32 * e];
                    v2[e] = Vs[(j + 2) * D + lane + 32 * e];
                    v3[e] = Vs[(j + 3) * D + lane + 32 * e];
                }
#pragma unroll
                for (int r = 0; r < RPW; ++r) {
                    const float4 p = *reinterpret_cast<const float4 *>(pw + r * kKT + j);
#pragma unroll
                    for (int e = 0; e < NV; ++e)
                        acc[r][e] = fmaf(p.x, v0[e], fmaf(p.y, v1[e], fmaf(p.z, v2[e], fmaf(p.w, v3[e], acc[r][e]))));
                }
            }
            __syncwarp();
        }
#pragma unroll
        for (int r = 0; r < RPW; ++r) {
            const int64_t at = u.base + (int64_t)cta * RT + warp * RPW + r;
            float sum = l[r];
#pragma unroll
            for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (r0 + warp * RPW + r < R) {
#pragma unroll
                for (int e = 0; e < NV; ++e) f.acc[at * D + lane + 32 * e] = acc[r][e];
                if (lane == 0) *reinterpret_cast<float2 *>(f.ml + at * 2) = make_float2(m[r], sum);
            }
        }
    }
    if (late) pdl_wait();
}

template <typename T, int NV, int RPW, int WARPS>
cudaError_t simt_launch(const PagedArgs *a, int fi, int late, int *ctas, cudaStream_t st) {
    auto kernel = paged_simt_kernel<T, NV, RPW, WARPS>;
    constexpr size_t smem = simt_smem<NV, RPW, WARPS>();
    static LaunchFit fit;
    const cudaError_t e = fit.prepare((const void *)kernel, WARPS * 32, smem, ctas);
    if (e != cudaSuccess || ctas) return e;
    return launch_pdl(kernel, a->f[fi].n, WARPS * 32, smem, st, *a, fi, late);
}

template <typename T, int RPW, int WARPS>
cudaError_t simt_by_d(int d, const PagedArgs *a, int fi, int late, int *ctas, cudaStream_t st) {
    switch (d / 32) {
        case 1: return simt_launch<T, 1, RPW, WARPS>(a, fi, late, ctas, st);
        case 2: return simt_launch<T, 2, RPW, WARPS>(a, fi, late, ctas, st);
        case 3: return simt_launch<T, 3, RPW, WARPS>(a, fi, late, ctas, st);
        case 4: return simt_launch<T, 4, RPW, WARPS>(a, fi, late, ctas, st);
        case 5: return simt_launch<T, 5, RPW, WARPS>(a, fi, late, ctas, st);
        case 6: return simt_launch<T, 6, RPW, WARPS>(a, fi, late, ctas, st);
        case 7: return simt_launch<T, 7, RPW, WARPS>(a, fi, late, ctas, st);
        case 8: return simt_launch<T, 8, RPW, WARPS>(a, fi, late, ctas, st);
        default: return cudaErrorInvalidValue;
    }
}

// ------------------------------------------------------------------ join
// A block per (token, KV head, up to 8 of its query heads), 8 / HB warps a head:
// the largest maximum M, the weights 2^(m - M), the weighted sums.  Own keys
// come first, then the prefix; warps' sums are added in order, so the result
// does not depend on timing.  Latency bound, so as much as can be is done ahead
// of the wait for the attention kernels (segments, plan, the places of the
// first 64 partials), and each warp's first sums are loaded beside the weights
// rather than behind them (one request of 8192 keys, 57 partials a head: 17.0
// -> 15.3 us).  A lane finds the weights of two partials and hands them to its
// warp.  Where tokens are few, a block has fewer heads and a head more warps,
// and registers for loads count; else blocks an SM do (64 registers: a prefix
// of 32768 keys for 64 requests 78.5 us, 96 registers 83.4).
constexpr int kJoinWarps = 8;

template <typename TOut, int HB, int NV>
__global__ void __launch_bounds__(kJoinWarps * 32, HB == 1 ? 2 : 4)
    paged_combine_kernel(const __grid_constant__ PagedArgs a) {
    constexpr int WPR = kJoinWarps / HB;  // warps a head
    __shared__ float4 sum[kJoinWarps][32 * NV];
    __shared__ int seg[2];
    __shared__ PagedParts parts[HB][2];
    __shared__ PlanShared plan[2];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int blocks = (a.G + HB - 1) / HB;  // of a token and KV head
    const int64_t t = blockIdx.x / (blocks * a.Hkv);
    const int hb = (int)(blockIdx.x - t * (blocks * a.Hkv)), h = hb / blocks, g0 = (hb - h * blocks) * HB;
    if (warp == 0) {
        // one token a sequence, no sequence without: token t is sequence t's
        int b = t < a.B && a.cu[t] <= t && t < a.cu[t + 1] ? (int)t : segment_of(a.cu + 1, a.B, t);
        if (b >= a.B || t < a.cu[b]) b = -1;  // behind the last sequence, or ahead of the first
        int g = -1;
        if (b >= 0 && a.n_groups > 0) {
            g = segment_of(a.groups + 1, a.n_groups, b);
            if (g >= a.n_groups || b < a.groups[g]) g = -1;  // a sequence outside every group
        }
        if (lane == 0) {
            seg[0] = b;
            seg[1] = g;
        }
    }
    __syncthreads();
    long long per[2] = {1, 1};
    if (a.here) {  // all places are found ahead of the wait for the attention kernels
        long long W;
        per[0] = paged_plan_here<kJoinWarps * 32>(a, a.f[0], 0, seg[0], plan[0], W);
        if (a.n_groups > 0) per[1] = paged_plan_here<kJoinWarps * 32>(a, a.f[1], 1, seg[1], plan[1], W);
    } else {
        pdl_wait();
        for (int i = 0; i < (a.n_groups > 0 ? 2 : 1); ++i) {
            per[i] = __ldcg(&a.f[i].hdr->err) ? 0 : __ldcg(&a.f[i].hdr->per);
            if ((int)threadIdx.x == i && seg[i] >= 0) plan[i].g = paged_seg(a.f[i], seg[i]);
        }
        __syncthreads();
    }
    const bool fine = seg[0] >= 0 && per[0] && per[1];  // (an array that is not as it must be: nothing is written)
    if (fine && threadIdx.x < 2 * HB && g0 + (int)threadIdx.x / 2 < a.G) {
        const int i = threadIdx.x & 1;
        const PagedSeg &sg = plan[i].g;
        parts[threadIdx.x / 2][i] = seg[i] < 0 ? PagedParts{}
                                               : paged_parts(a, a.f[i], sg, i ? per[1] : per[0],
                                                             (int)(t - sg.tok0) * a.G + g0 + (int)threadIdx.x / 2, h);
    }
    __syncthreads();
    const int sub = warp % WPR, g = g0 + warp / WPR, d4 = a.d / 4;
    const bool live = fine && g < a.G;
    const int own = live ? parts[warp / WPR][0].cnt : 0, cnt = live ? own + parts[warp / WPR][1].cnt : 0;
    // lane's partials i0 + lane and i0 + lane + 32: their (m, l) and sums
    const float2 *ml[2];
    const float *src[2];
    auto place = [&](int i0) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            int i = i0 + 32 * u + lane;
            const int fi = i < own ? 0 : 1;
            ml[u] = nullptr;
            src[u] = nullptr;
            if (fi) i -= own;
            const long long row = paged_part(a.f[fi], parts[warp / WPR][fi], fi ? per[1] : per[0], i);
            if (row >= 0) {
                ml[u] = reinterpret_cast<const float2 *>(a.f[fi].ml) + row;
                src[u] = a.f[fi].acc + row * a.d;
            }
        }
    };
    auto at_lane = [&](const float *p, int k) {
        return reinterpret_cast<const float4 *>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(p), k));
    };
    if (cnt > 0) place(0);
    if (a.here) pdl_wait();
    if (!fine) return;
    float M = -INFINITY, L = 0.f;
    float4 o[NV];
#pragma unroll
    for (int e = 0; e < NV; ++e) o[e] = make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int PRE = 4 / NV;  // sums of a warp that are loaded beside the weights, not behind them
    // the maximum is carried along, as in the attention itself: 64 partials a trip
#pragma unroll 1
    for (int i0 = 0; i0 < cnt; i0 += 64) {
        if (i0) place(i0);
        const int most = min(64, cnt - i0);
        float2 v[2];
        float4 x[PRE][NV];
#pragma unroll
        for (int u = 0; u < 2; ++u) v[u] = ml[u] ? __ldcg(ml[u]) : make_float2(-INFINITY, 0.f);
#pragma unroll
        for (int j = 0; j < PRE; ++j) {
            const int u = j * WPR / 32, k = sub + j * WPR;  // (u: a constant, sub < WPR)
            const float4 *q = at_lane(src[u], k & 31);
#pragma unroll
            for (int e = 0; e < NV; ++e)
                if (u < 2 && k < most && q && lane + 32 * e < d4) x[j][e] = __ldcg(q + lane + 32 * e);
        }
        float Mn = M;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            if (v[u].y != v[u].y) v[u].x = INFINITY;  // NaN scores leave no maximum: the row is to become NaN, not empty
            Mn = fmaxf(Mn, v[u].x);
        }
#pragma unroll
        for (int s = 16; s; s >>= 1) Mn = fmaxf(Mn, __shfl_xor_sync(0xffffffffu, Mn, s));
        if (Mn == -INFINITY) continue;
        const float alpha = exp2f(M - Mn);
        float w[2];
        M = Mn;
        L *= alpha;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            w[u] = exp2f(v[u].x - Mn);
            L += w[u] * v[u].y;
        }
#pragma unroll
        for (int e = 0; e < NV; ++e) {
            o[e].x *= alpha;
            o[e].y *= alpha;
            o[e].z *= alpha;
            o[e].w *= alpha;
        }
        // (a partial without weight may never have been written)
        auto add = [&](float wk, const float4 &y, float4 &z) {
            z.x = fmaf(wk, y.x, z.x);
            z.y = fmaf(wk, y.y, z.y);
            z.z = fmaf(wk, y.z, z.z);
            z.w = fmaf(wk, y.w, z.w);
        };
#pragma unroll
        for (int j = 0; j < PRE; ++j) {
            const int u = j * WPR / 32, k = sub + j * WPR;
            const float wk = __shfl_sync(0xffffffffu, w[u], k & 31);
#pragma unroll
            for (int e = 0; e < NV; ++e)
                if (u < 2 && k < most && wk != 0.f && lane + 32 * e < d4) add(wk, x[j][e], o[e]);
        }
#pragma unroll 4
        for (int k = sub + PRE * WPR; k < most; k += WPR) {
            const float w0 = __shfl_sync(0xffffffffu, w[0], k & 31), w1 = __shfl_sync(0xffffffffu, w[1], k & 31);
            const float4 *q0 = at_lane(src[0], k & 31), *q1 = at_lane(src[1], k & 31);
            const float wk = k < 32 ? w0 : w1;
            const float4 *q = k < 32 ? q0 : q1;
#pragma unroll
            for (int e = 0; e < NV; ++e)
                if (wk != 0.f && lane + 32 * e < d4) add(wk, __ldcg(q + lane + 32 * e), o[e]);
        }
    }
#pragma unroll
    for (int s = 16; s; s >>= 1) L += __shfl_xor_sync(0xffffffffu, L, s);
    if (WPR > 1) {
#pragma unroll
        for (int e = 0; e < NV; ++e) sum[warp][lane + 32 * e] = o[e];
        __syncthreads();
    }
    if (!live) return;
    const float inv = L == 0.f ? 0.f : 1.f / L;  // (0: no visible key)
    const int head = h * a.G + g;
    TOut *out = static_cast<TOut *>(a.out) + (t * a.Hq + head) * a.d;
#pragma unroll
    for (int e = 0; e < NV; ++e) {
        const int c = lane + 32 * e;
        if (c >= d4 || (WPR > 1 && sub != e)) continue;  // (of several warps, warp e of the head writes vector e)
        float4 v = o[e];
        if (WPR > 1) {
            v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int i = 0; i < WPR; ++i) {
                const float4 x = sum[warp - sub + i][c];
                v.x += x.x;
                v.y += x.y;
                v.z += x.z;
                v.w += x.w;
            }
        }
        if constexpr (sizeof(TOut) == 4) {
            *reinterpret_cast<float4 *>(out + c * 4) = make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
        } else {
            uint2 pk;
            pk.x = pack_bf16x2(v.x * inv, v.y * inv);
            pk.y = pack_bf16x2(v.z * inv, v.w * inv);
            *reinterpret_cast<uint2 *>(out + c * 4) = pk;
        }
    }
    if (sub == 0 && lane == 0)
        a.lse[(int64_t)head * a.T + t] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.69314718055994531f;
}

template <typename TOut, int NV>
cudaError_t combine_as(const PagedArgs &a, cudaStream_t st) {
    // heads a block: as many as it takes to leave every SM two blocks
    auto blocks = [&](int hb) { return a.T * a.Hkv * ((a.G + hb - 1) / hb); };  // < 2^31
    int hb = 1;
    while (hb < 8 && hb < a.G && blocks(2 * hb) >= 2 * paged_sms()) hb *= 2;
    auto go = [&](auto kernel) { return launch_pdl(kernel, (unsigned)blocks(hb), kJoinWarps * 32, 0, st, a); };
    return hb == 1   ? go(paged_combine_kernel<TOut, 1, NV>)
           : hb == 2 ? go(paged_combine_kernel<TOut, 2, NV>)
           : hb == 4 ? go(paged_combine_kernel<TOut, 4, NV>)
                     : go(paged_combine_kernel<TOut, 8, NV>);
}

}  // namespace

cudaError_t launch_paged_plan(const PagedArgs &a, cudaStream_t st) {
    paged_plan_kernel<<<a.n_groups > 0 ? 2 : 1, kPlanThreads, 0, st>>>(a);
    return cudaGetLastError();
}

int paged_sms() {
    static std::atomic<int> sms[128] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 128) return 1;
    int n = sms[dev].load(std::memory_order_relaxed);
    if (!n) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = 1;
        sms[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

int paged_simt_ctas(int rt, int d) {
    int n = 0;
    const cudaError_t e = rt == 16 ? simt_by_d<float, 4, 4>(d, nullptr, 0, 0, &n, nullptr)
                                   : simt_by_d<float, 8, 8>(d, nullptr, 0, 0, &n, nullptr);
    if (e != cudaSuccess || n < 1) n = 1;
    return std::min(kPagedMaxCtas, n * paged_sms());
}

cudaError_t launch_paged_simt(const PagedArgs &a, int fi, int late, cudaStream_t st) {
    const bool few = a.f[fi].rt == 16;
    if (a.dtype == RA_FP32)
        return few ? simt_by_d<float, 4, 4>(a.d, &a, fi, late, nullptr, st)
                   : simt_by_d<float, 8, 8>(a.d, &a, fi, late, nullptr, st);
    return few ? simt_by_d<__nv_bfloat16, 4, 4>(a.d, &a, fi, late, nullptr, st)
               : simt_by_d<__nv_bfloat16, 8, 8>(a.d, &a, fi, late, nullptr, st);
}

cudaError_t launch_paged_combine(const PagedArgs &a, cudaStream_t st) {
    if (a.out_dtype == RA_FP32) return a.d <= 128 ? combine_as<float, 1>(a, st) : combine_as<float, 2>(a, st);
    return a.d <= 128 ? combine_as<__nv_bfloat16, 1>(a, st) : combine_as<__nv_bfloat16, 2>(a, st);
}

}  // namespace ra

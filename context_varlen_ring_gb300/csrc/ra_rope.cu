// ra_rope.cu -- rotary positions (forward and gradient) and the paged-cache
// append that rotates on the way.  One kernel serves both: a list of jobs
// (queries, keys, values), each rotated or copied, each written to token rows
// or to the cache row of its token.
//
// Mathematics: pair i of token t turns by phi = pos[axis_i][t] * f_i.  The
// table holds f_i / (2 pi) as a 64-bit fraction of a turn, so pos * turns
// modulo 2^64 is the angle modulo a full turn, without any rounding that grows with the
// position, in one 64-bit integer product; its upper 32 bits, as a signed
// fraction of half a turn, go through sincospif.
//
// Bound: memory.  Per token (Hq + Hk) * d elements are read and written; the
// n_pairs sines and cosines are computed once per token into shared memory
// and used by every head.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "ra_dev.cuh"
#include "ra_kernels.h"

namespace ra {
namespace {

template <typename T, int VEC>
struct Pack;
template <>
struct Pack<__nv_bfloat16, 8> {
    using V = uint4;
};
template <>
struct Pack<float, 4> {
    using V = uint4;
};
template <>
struct Pack<__nv_bfloat16, 1> {
    using V = unsigned short;
};
template <>
struct Pack<float, 1> {
    using V = uint32_t;
};

template <typename T, int VEC>
__device__ __forceinline__ void unpack(const typename Pack<T, VEC>::V &v, float (&f)[VEC]) {
    const T *e = reinterpret_cast<const T *>(&v);
#pragma unroll
    for (int i = 0; i < VEC; ++i) f[i] = (float)e[i];
}
template <typename T, int VEC>
__device__ __forceinline__ typename Pack<T, VEC>::V repack(const float (&f)[VEC]) {
    typename Pack<T, VEC>::V v;
    T *e = reinterpret_cast<T *>(&v);
#pragma unroll
    for (int i = 0; i < VEC; ++i) e[i] = (T)f[i];  // round to nearest even: the one rounding of the result
    return v;
}

// A block owns TT tokens; thread (u, hs) owns unit u (a vector, or the two
// vectors of a half-split pair) of heads hs, hs + hpb, ...  Its sines and
// cosines are those of unit u for every head, and the TT tokens' vectors are
// loaded before the angles are computed, so TT (x 2) 16-byte loads per thread
// hide behind the table work.
template <typename T, int VEC, bool ADJ, int TT>
__global__ void __launch_bounds__(1024) rope_kernel(const __grid_constant__ RopeParams p) {
    using V = typename Pack<T, VEC>::V;
    extern __shared__ float2 cs[];  // [TT][n_pairs]: cos, sin
    __shared__ long long row_off[TT];
    __shared__ int row_ok[TT];      // 0: leave the token alone, 1: its token rows only, 2: its cache row too
    const int64_t t0 = (int64_t)blockIdx.x * TT;
    const int u = threadIdx.x % p.units, hs = threadIdx.x / p.units;
    const bool rot = u < p.rot_units;
    int off0, off1 = -1, pb = 0;
    if (!rot) {
        off0 = 2 * p.n_pairs + (u - p.rot_units) * VEC;
    } else if (VEC > 1 && ADJ) {
        off0 = u * VEC;
        pb = u * (VEC / 2);
    } else if (VEC == 1 && p.adjacent) {
        off0 = 2 * u;
        off1 = 2 * u + 1;
        pb = u;
    } else {
        off0 = u * VEC;
        off1 = p.n_pairs + u * VEC;
        pb = u * VEC;
    }

    bool first = true;
    for (int h = hs;; h += p.heads_per_block) {
        // every thread makes the first trip (it holds the barrier); later
        // trips are taken by the threads that have a head left
        const bool have = h < p.total_heads && hs < p.heads_per_block;
        int j = 0, hl = h;
        if (have) {
            while (hl >= p.jobs[j].heads) hl -= p.jobs[j++].heads;
        }
        const RopeJob &job = p.jobs[have ? j : 0];
        V a[TT], b[TT];
        if (have) {
            const T *x = static_cast<const T *>(job.x) + (int64_t)hl * p.d;
#pragma unroll
            for (int i = 0; i < TT; ++i) {
                if (t0 + i < p.T) {
                    const T *r = x + (t0 + i) * job.x_stride;
                    a[i] = *reinterpret_cast<const V *>(r + off0);
                    if (off1 >= 0) b[i] = *reinterpret_cast<const V *>(r + off1);
                }
            }
        }
        if (first) {
            first = false;
            const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = (blockDim.x + 31) >> 5;
            if (p.cu) {
                // the sequence of each token: the number of segment ends <= t
                for (int i = warp; i < TT; i += warps) {
                    const int64_t t = t0 + i;
                    int ok = 0;
                    long long off = 0;
                    if (t < p.T) {
                        const int s = dev::segment_of(p.cu + 1, p.B, t);
                        if (s < p.B) {
                            const long long c0 = p.cu[s], n = (long long)p.cu[s + 1] - c0;
                            const long long idx = (long long)p.kv_lens[s] - n + (t - c0);
                            ok = 1;
                            bool in = t >= c0 && idx >= 0 && idx < p.table_width * p.page_size;
                            if (in) {
                                const int pg = p.page_table[(int64_t)s * p.table_width + idx / p.page_size];
                                in = pg >= 0 && pg < p.n_pages;
                                off = pg * p.page_stride + (idx % p.page_size) * p.token_stride;
                            }
                            if (in)
                                ok = 2;
                            else if (lane == 0)
                                dev::record_status(p.status, RA_ERR_DEVICE_BOUNDS);
                        }
                    }
                    if (lane == 0) {
                        row_ok[i] = ok;
                        row_off[i] = off;
                    }
                }
            } else if (threadIdx.x < TT) {
                row_ok[threadIdx.x] = t0 + threadIdx.x < p.T ? 1 : 0;
            }
            for (int w = threadIdx.x; w < TT * p.n_pairs; w += blockDim.x) {
                const int i = w / p.n_pairs, pr = w - i * p.n_pairs;
                if (t0 + i < p.T) {
                    const long long pos = p.pos[(int64_t)p.axis[pr] * p.T + t0 + i];
                    const unsigned long long turn = (unsigned long long)pos * p.turns[pr];
                    // the upper half as a signed number of 2^-31 half turns
                    float s, c;
                    sincospif((float)(int)(turn >> 32) * 4.6566128730773926e-10f, &s, &c);
                    cs[w] = make_float2(c, p.inverse ? -s : s);
                }
            }
            __syncthreads();
        }
        if (!have) break;
        T *y0 = static_cast<T *>(job.y) + (job.paged ? (int64_t)hl * p.head_stride : (int64_t)hl * p.d);
        const bool turn = rot && job.rotate;
        if (job.x == job.y && !turn) continue;  // in place and passed through
#pragma unroll
        for (int i = 0; i < TT; ++i) {
            if (row_ok[i] < (job.paged ? 2 : 1)) continue;
            T *y = y0 + (job.paged ? (int64_t)row_off[i] : (t0 + i) * job.y_stride);
            if (turn) {
                const float2 *t = cs + i * p.n_pairs + pb;
                float fa[VEC], fb[VEC];
                unpack<T, VEC>(a[i], fa);
                if (VEC > 1 && ADJ) {
#pragma unroll
                    for (int e = 0; e + 1 < VEC; e += 2) {
                        const float2 r = t[e / 2];
                        const float x0 = fa[e], x1 = fa[e + 1];
                        fa[e] = x0 * r.x - x1 * r.y;
                        fa[e + 1] = x0 * r.y + x1 * r.x;
                    }
                } else {
                    unpack<T, VEC>(b[i], fb);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        const float2 r = t[e];
                        const float x0 = fa[e], x1 = fb[e];
                        fa[e] = x0 * r.x - x1 * r.y;
                        fb[e] = x0 * r.y + x1 * r.x;
                    }
                    b[i] = repack<T, VEC>(fb);
                }
                a[i] = repack<T, VEC>(fa);
            }
            *reinterpret_cast<V *>(y + off0) = a[i];
            if (off1 >= 0) *reinterpret_cast<V *>(y + off1) = b[i];
        }
    }
}

template <typename T, int VEC, bool ADJ>
cudaError_t launch_tt(const RopeParams &p, int threads, int tt, cudaStream_t st) {
    const size_t smem = (size_t)tt * p.n_pairs * sizeof(float2);
    const unsigned grid = (unsigned)((p.T + tt - 1) / tt);
    if (tt == 4)
        rope_kernel<T, VEC, ADJ, 4><<<grid, threads, smem, st>>>(p);
    else
        rope_kernel<T, VEC, ADJ, 1><<<grid, threads, smem, st>>>(p);
    return cudaGetLastError();
}

}  // namespace

void rope_table(RopeParams &p, const double *inv_freq, const uint8_t *axes, int n_pairs, int adjacent, int inverse) {
    p.n_pairs = n_pairs;
    p.adjacent = adjacent ? 1 : 0;
    p.inverse = inverse;
    for (int i = 0; i < n_pairs; ++i) {
        const double turns = inv_freq[i] * 0.15915494309189533577;  // 1 / (2 pi)
        const double frac = turns - std::floor(turns);              // in [0, 1]
        p.turns[i] = frac >= 1.0 ? 0ull : (uint64_t)std::ldexp(frac, 64);
        p.axis[i] = axes ? axes[i] : 0;
    }
}

cudaError_t launch_rope(RopeParams &p, int dtype, cudaStream_t st) {
    if (p.T <= 0) return cudaSuccess;
    const int es = dtype == RA_FP32 ? 4 : 2;
    int vec = 16 / es;
    // the 16-byte path: every row, head and unit starts on 16 bytes
    bool fast = p.d % vec == 0 && (p.adjacent ? 2 * p.n_pairs : p.n_pairs) % vec == 0;
    p.total_heads = 0;
    for (int j = 0; j < p.njobs; ++j) {
        const RopeJob &jb = p.jobs[j];
        p.total_heads += jb.heads;
        fast = fast && !(reinterpret_cast<uintptr_t>(jb.x) % 16) && !(reinterpret_cast<uintptr_t>(jb.y) % 16) &&
               jb.x_stride % vec == 0 && jb.y_stride % vec == 0;
        if (jb.paged)
            fast = fast && p.page_stride % vec == 0 && p.token_stride % vec == 0 && p.head_stride % vec == 0;
    }
    if (!fast) vec = 1;
    const bool adj = fast && p.adjacent;
    p.rot_units = adj ? 2 * p.n_pairs / vec : p.n_pairs / vec;
    p.units = p.rot_units + (p.d - 2 * p.n_pairs) / vec;
    const int trips = (p.total_heads * p.units + 639) / 640;
    p.heads_per_block = std::max(1, (p.total_heads + trips - 1) / trips);
    const int threads = std::min(1024, (p.units * p.heads_per_block + 31) / 32 * 32);
    const int tt = p.T >= 1216 ? 4 : 1;
    if (dtype == RA_FP32) {
        if (!fast) return launch_tt<float, 1, false>(p, threads, tt, st);
        return adj ? launch_tt<float, 4, true>(p, threads, tt, st) : launch_tt<float, 4, false>(p, threads, tt, st);
    }
    if (!fast) return launch_tt<__nv_bfloat16, 1, false>(p, threads, tt, st);
    return adj ? launch_tt<__nv_bfloat16, 8, true>(p, threads, tt, st)
               : launch_tt<__nv_bfloat16, 8, false>(p, threads, tt, st);
}

}  // namespace ra

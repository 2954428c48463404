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

constexpr int kRopeWarps = 4;

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

// A warp owns a token, or where tokens are few every S-th group of its heads.
// Lane (hh, u) owns unit u (a vector, or the two vectors of a half-split pair)
// of heads hh, hh + hpi, ...: its sines and cosines stay in registers for all
// of them, so shared memory carries each angle once a token (with a read per
// head the shared-memory pipe was the limit, at 81 %: 134 us for 32768 tokens
// of 40 heads of 128 and 90 us for 8192 of 72; this form takes 128 and 64 us).
// Two heads a lane are in flight, the first two before the angles are
// computed; eight blocks an SM beat five with four heads in flight (131 us)
// and ten that spill (164 us).
template <typename T, int VEC, bool ADJ>
__global__ void __launch_bounds__(kRopeWarps * 32, 8) rope_kernel(const __grid_constant__ RopeParams p) {
    using V = typename Pack<T, VEC>::V;
    constexpr int UN = 2, NP = VEC > 1 && ADJ ? VEC / 2 : VEC;  // heads in flight, pairs a unit
    extern __shared__ float2 cs_all[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float2 *cs = cs_all + warp * p.n_pairs;
    const int64_t gw = (int64_t)blockIdx.x * kRopeWarps + warp;
    const int64_t t = gw / p.split;
    if (t >= p.T) return;
    const int sub = (int)(gw - t * p.split);

    bool first = true;
    int ok = 1;          // 0: leave the token alone, 1: its token rows only, 2: its cache row too
    long long off = 0;   // its cache row
    auto prepare = [&]() {
        if (p.cu) {
            // the token's sequence: the number of segment ends <= t
            const int s = dev::segment_of(p.cu + 1, p.B, t);
            ok = 0;
            if (s < p.B) {
                const long long c0 = p.cu[s], n = (long long)p.cu[s + 1] - c0;
                const long long idx = (long long)p.kv_lens[s] - n + (t - c0);
                bool in = t >= c0 && idx >= 0 && idx < p.table_width * p.page_size;
                if (in) {
                    const int pg = p.page_table[(int64_t)s * p.table_width + (int)idx / p.page_size];
                    in = pg >= 0 && pg < p.n_pages;
                    off = pg * p.page_stride + ((int)idx % p.page_size) * p.token_stride;
                }
                ok = in ? 2 : 1;
                if (!in && lane == 0) dev::record_status(p.status, RA_ERR_DEVICE_BOUNDS);
            }
        }
        for (int w = lane; w < p.n_pairs; w += 32) {
            const long long pos = p.pos[(int64_t)p.axis[w] * p.T + t];
            const unsigned long long turn = (unsigned long long)pos * p.turns[w];
            // the upper half as a signed number of 2^-31 half turns
            float s, c;
            sincospif((float)(int)(turn >> 32) * 4.6566128730773926e-10f, &s, &c);
            cs[w] = make_float2(c, p.inverse ? -s : s);
        }
        __syncwarp();
    };
    for (int u0 = 0; u0 < p.units; u0 += 32) {  // (one trip unless a head has more than 32 units)
        const int hpi = p.units > 32 ? 1 : 32 / p.units;
        const int hh = p.units > 32 ? 0 : lane / p.units, u = p.units > 32 ? u0 + lane : lane % p.units;
        const bool mine = hh < hpi && u < p.units;
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
        float2 r[NP];
        bool loaded = false;
        int skip = sub;  // groups of heads ahead of this warp's first in the next job
        for (int j = 0; j < p.njobs; ++j) {
            const RopeJob &jb = p.jobs[j];
            const int heads = mine ? jb.heads - hh : 0, step = p.split * hpi;  // heads from this lane's on
            const T *x = static_cast<const T *>(jb.x) + t * jb.x_stride + hh * p.d;
            const bool turn = rot && jb.rotate;
            const int groups = (jb.heads + hpi - 1) / hpi;
            int h = skip * hpi;
            while (skip < groups) skip += p.split;
            skip -= groups;
            for (; h < jb.heads; h += UN * step) {
                V a[UN], b[UN];
#pragma unroll
                for (int i = 0; i < UN; ++i) {
                    if (h + i * step < heads) {
                        a[i] = *reinterpret_cast<const V *>(x + (h + i * step) * p.d + off0);
                        if (off1 >= 0) b[i] = *reinterpret_cast<const V *>(x + (h + i * step) * p.d + off1);
                    }
                }
                if (first) {
                    first = false;
                    prepare();
                }
                if (!loaded) {
                    loaded = true;
                    if (rot && mine) {
#pragma unroll
                        for (int e = 0; e < NP; ++e) r[e] = cs[pb + e];
                    }
                }
                if (ok < (jb.paged ? 2 : 1) || (jb.x == jb.y && !turn)) continue;  // (in place and passed through)
                T *y = static_cast<T *>(jb.y) + (jb.paged ? off : t * jb.y_stride);
                const int64_t hs = jb.paged ? p.head_stride : p.d;
#pragma unroll
                for (int i = 0; i < UN; ++i) {
                    if (h + i * step >= heads) continue;
                    if (turn) {
                        float fa[VEC], fb[VEC];
                        unpack<T, VEC>(a[i], fa);
                        if (VEC > 1 && ADJ) {
#pragma unroll
                            for (int e = 0; e < NP; ++e) {
                                const float x0 = fa[(2 * e) % VEC], x1 = fa[(2 * e + 1) % VEC];
                                fa[(2 * e) % VEC] = x0 * r[e].x - x1 * r[e].y;
                                fa[(2 * e + 1) % VEC] = x0 * r[e].y + x1 * r[e].x;
                            }
                        } else {
                            unpack<T, VEC>(b[i], fb);
#pragma unroll
                            for (int e = 0; e < VEC; ++e) {
                                const float x0 = fa[e], x1 = fb[e];
                                fa[e] = x0 * r[e % NP].x - x1 * r[e % NP].y;
                                fb[e] = x0 * r[e % NP].y + x1 * r[e % NP].x;
                            }
                            b[i] = repack<T, VEC>(fb);
                        }
                        a[i] = repack<T, VEC>(fa);
                    }
                    T *yh = y + (h + i * step + hh) * hs;
                    *reinterpret_cast<V *>(yh + off0) = a[i];
                    if (off1 >= 0) *reinterpret_cast<V *>(yh + off1) = b[i];
                }
            }
        }
    }
}

template <typename T, int VEC, bool ADJ>
cudaError_t launch_warps(const RopeParams &p, cudaStream_t st) {
    const size_t smem = (size_t)kRopeWarps * p.n_pairs * sizeof(float2);
    const int64_t blocks = (p.T * p.split + kRopeWarps - 1) / kRopeWarps;
    rope_kernel<T, VEC, ADJ><<<(unsigned)blocks, kRopeWarps * 32, smem, st>>>(p);
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
    // warps a token: enough to fill the GPU (16 warps an SM) when tokens are few, at most one per group of heads
    const int groups = p.units > 32 ? p.total_heads : (p.total_heads + 32 / p.units - 1) / (32 / p.units);
    p.split = (int)std::min<int64_t>(groups, std::max<int64_t>(1, 152 * 16 / p.T));
    if (dtype == RA_FP32) {
        if (!fast) return launch_warps<float, 1, false>(p, st);
        return adj ? launch_warps<float, 4, true>(p, st) : launch_warps<float, 4, false>(p, st);
    }
    if (!fast) return launch_warps<__nv_bfloat16, 1, false>(p, st);
    return adj ? launch_warps<__nv_bfloat16, 8, true>(p, st) : launch_warps<__nv_bfloat16, 8, false>(p, st);
}

}  // namespace ra

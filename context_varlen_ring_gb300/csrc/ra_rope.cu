// ra_rope.cu -- rotary positions (forward and gradient) and the paged-cache
// append that rotates on the way.  One kernel serves both: a list of jobs
// (queries, keys, values), each rotated or copied, each written to token rows
// or to the cache row of its token.
//
// Mathematics: pair i of token t turns by phi = pos[axis_i][t] * f_i.  The
// table holds f_i / (2 pi) as a 64-bit fraction of a turn, so pos * turns
// modulo 2^64 is the angle modulo a full turn, without any rounding that grows with the
// position, in one 64-bit integer product; its distance to the nearest quarter
// turn goes through sincospif.
//
// Bound: memory.  Per token (Hq + Hk) * d elements are read and written; the
// n_pairs sines and cosines are computed once per token, meet in shared memory,
// and stay in registers for all heads.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "ra_kernels.h"
#include "ra_serve.cuh"

namespace ra {
namespace {

constexpr int kRopeWarps = 4;
constexpr int kBulkWarps = 16, kBulkStages = 8, kRingBytes = 212 * 1024, kBulkSmem = 224 * 1024;
constexpr int kHeldWarps = 20;

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

// The rotation of one unit, the same arithmetic in both kernels below: a
// product, rounded, and a fused product and sum.  Half-split pairs: two
// vectors; neighbouring pairs: one, with half as many angles.
template <typename T, int VEC, bool ADJ, int NP>
__device__ __forceinline__ void turn_unit(typename Pack<T, VEC>::V &a, typename Pack<T, VEC>::V &b,
                                          const float (&c)[NP], const float (&s)[NP]) {
    float fa[VEC], fb[VEC];
    unpack<T, VEC>(a, fa);
    if (VEC > 1 && ADJ) {
#pragma unroll
        for (int e = 0; e < NP; ++e) {
            const float x = fa[(2 * e) % VEC], y = fa[(2 * e + 1) % VEC];
            fa[(2 * e) % VEC] = fmaf(x, c[e], -__fmul_rn(y, s[e]));
            fa[(2 * e + 1) % VEC] = fmaf(x, s[e], __fmul_rn(y, c[e]));
        }
    } else {
        unpack<T, VEC>(b, fb);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const float x = fa[e], y = fb[e];
            fa[e] = fmaf(x, c[e % NP], -__fmul_rn(y, s[e % NP]));
            fb[e] = fmaf(x, s[e % NP], __fmul_rn(y, c[e % NP]));
        }
        b = repack<T, VEC>(fb);
    }
    a = repack<T, VEC>(fa);
}

// Cosine and sine of pos * turns / 2^64 of a turn.  The upper two bits of the
// angle, rounded, are its quarter; what is left of it, an eighth of a turn at
// most either way, becomes a float of 2^-33 half turns (that of a whole angle
// would be off by 2^-25 half turns, four times as much).
__device__ __forceinline__ float2 angle(int pos, unsigned long long turns, int inverse) {
    const unsigned long long turn = (unsigned long long)(long long)pos * turns;
    const unsigned hi = (unsigned)(turn >> 32), quarter = (hi + 0x20000000u) >> 30;
    const int rest = (int)__funnelshift_l((unsigned)turn, hi, 2);
    float s, c;
    sincospif((float)rest * 1.1641532182693481e-10f, &s, &c);
    const bool odd = quarter & 1;
    // (quarters 1 and 2 negate the cosine, 2 and 3 the sine, the gradient the sine once more)
    return make_float2(__uint_as_float(__float_as_uint(odd ? s : c) ^ ((quarter + 1) & 2) << 30),
                       __uint_as_float(__float_as_uint(odd ? c : s) ^ ((quarter ^ (unsigned)inverse << 1) & 2) << 30));
}

__device__ __forceinline__ int page_of(const RopeParams &p, int key) {
    return p.page_shift >= 0 ? key >> p.page_shift : key / p.page_size;
}

// A warp owns a token, or where tokens are few every S-th group of its heads.
// Lane (hh, u) owns unit u (a vector, or the two vectors of a half-split pair)
// of heads hh, hh + hpi, ...: its sines and cosines stay in registers for all
// of them, so shared memory carries each angle once a token (with a read per
// head the shared-memory pipe was the limit, at 81 %).  Two heads a lane are
// in flight, the first two before the angles are computed.  A chain of loads
// bounds the small calls this kernel is for (64 tokens appended to their
// caches: 5.1 us): the token's sequence, its page, and beside them the positions.
template <typename T, int VEC, bool ADJ>
__global__ void __launch_bounds__(kRopeWarps * 32, 4) rope_kernel(const __grid_constant__ RopeParams p) {
    using V = typename Pack<T, VEC>::V;
    constexpr int UN = 2, NP = VEC > 1 && ADJ ? VEC / 2 : VEC;  // heads in flight, pairs a unit
    extern __shared__ float2 cs_all[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float2 *cs = cs_all + warp * p.n_pairs;
    const int64_t gw = (int64_t)blockIdx.x * kRopeWarps + warp;
    const int64_t t = p.split == 1 ? gw : (int64_t)((unsigned)gw / (unsigned)p.split);  // (split only when tokens are few)
    if (t >= p.T) return;
    const int sub = (int)(gw - t * p.split);

    bool first = true;
    int ok = 1;          // 0: leave the token alone, 1: its token rows only, 2: its cache row too
    long long off = 0;   // its cache row
    auto prepare = [&]() {
        int pos[4];  // of this lane's pairs, in flight beside the search
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int w = lane + 32 * k;
            if (w < p.n_pairs) pos[k] = __ldg(p.pos + (int64_t)p.axis[w] * p.T + t);
        }
        if (p.cu) {
            // the token's sequence: token t's is t in a decoding step, else the number of segment ends <= t
            int s = p.B;
            if (t < p.B && p.cu[t] <= t && t < p.cu[t + 1])
                s = (int)t;
            else
                s = dev::segment_of(p.cu + 1, p.B, t);
            ok = 0;
            if (s < p.B) {
                const long long c0 = p.cu[s], n = (long long)p.cu[s + 1] - c0;
                const long long idx = (long long)p.kv_lens[s] - n + (t - c0);
                bool in = t >= c0 && idx >= 0 && idx < p.table_keys;
                if (in) {
                    const int pi = page_of(p, (int)idx);
                    const int pg = p.page_table[(int64_t)s * p.table_width + pi];
                    in = pg >= 0 && pg < p.n_pages;
                    off = pg * p.page_stride + ((int)idx - pi * p.page_size) * p.token_stride;
                }
                ok = in ? 2 : 1;
                if (!in && lane == 0) dev::record_status(p.status, RA_ERR_DEVICE_BOUNDS);
            }
        }
#pragma unroll 1
        for (int k = 0; 32 * k < p.n_pairs; ++k) {
            const int w = lane + 32 * k;
            if (w < p.n_pairs) {
                const int at = k == 0 ? pos[0] : k == 1 ? pos[1] : k == 2 ? pos[2] : pos[3];
                cs[w] = angle(at, p.turns[w], p.inverse);
            }
        }
        __syncwarp();
    };
    for (int u0 = 0; u0 < p.units; u0 += 32) {  // (one trip unless a head has more than 32 units)
        const int hpi = p.hpi;
        const int hh = p.units > 32 ? 0 : lane * p.unit_inv >> 16, u = u0 + lane - hh * p.units;
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
        float rc[NP], rs[NP];
        bool loaded = false;
        int skip = sub;  // groups of heads ahead of this warp's first in the next job
        for (int j = 0; j < p.njobs; ++j) {
            const RopeJob &jb = p.jobs[j];
            const int heads = mine ? jb.heads - hh : 0, step = p.split * hpi;  // heads from this lane's on
            const T *x = static_cast<const T *>(jb.x) + t * jb.x_stride + hh * p.d;
            const bool turn = rot && jb.rotate;
            const int groups = jb.groups;
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
                        for (int e = 0; e < NP; ++e) {
                            const float2 r = cs[pb + e];
                            rc[e] = r.x;
                            rs[e] = r.y;
                        }
                    }
                }
                if (ok < (jb.paged ? 2 : 1) || (jb.x == jb.y && !turn)) continue;  // (in place and passed through)
                T *y = static_cast<T *>(jb.y) + (jb.paged ? off : t * jb.y_stride);
                const int64_t hs = jb.paged ? p.head_stride : p.d;
#pragma unroll
                for (int i = 0; i < UN; ++i) {
                    if (h + i * step >= heads) continue;
                    if (turn) turn_unit<T, VEC, ADJ, NP>(a[i], b[i], rc, rs);
                    T *yh = y + (h + i * step + hh) * hs;
                    *reinterpret_cast<V *>(yh + off0) = a[i];
                    if (off1 >= 0) *reinterpret_cast<V *>(yh + off1) = b[i];
                }
            }
        }
    }
}

// The same for many tokens: each warp streams its tokens through a ring in
// shared memory, copied in and out by the bulk-copy engine.  All warps go
// through the tokens side by side (with a run of consecutive tokens each, their
// rows lay at multiples of one distance and met in the same memory channels:
// 112 to 130 us for 32768 tokens, 104 to 107 so).
// A stage holds a token's heads (queries, keys, values, one behind the other),
// or one of `parts` shares of them; the rotated units are read, turned and
// written back in place.  So the bytes in flight are the rings' (some 100 KB
// an SM) and no thread's registers wait for memory.
template <typename T, bool ADJ>
__global__ void __launch_bounds__(kBulkWarps * 32) rope_bulk_kernel(const __grid_constant__ RopeParams p) {
    constexpr int VEC = 16 / (int)sizeof(T), NP = ADJ ? VEC / 2 : VEC;
    using V = typename Pack<T, VEC>::V;
    extern __shared__ __align__(128) uint8_t smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    uint8_t *ring = smem + (size_t)warp * p.stages * p.stage_bytes;
    float2 *cs = reinterpret_cast<float2 *>(smem + (size_t)warps * p.stages * p.stage_bytes) + warp * p.n_pairs;
    __shared__ uint64_t full[kBulkWarps][kBulkStages];
    __shared__ int abort_flag;
    if (threadIdx.x == 0) abort_flag = 0;
    if (lane == 0) {
        for (int i = 0; i < p.stages; ++i) dev::mbar_init(&full[warp][i], 1);
        dev::fence_mbar_init();
    }
    __syncthreads();
    const dev::WaitCtl wc{&abort_flag, p.status, p.budget_ns};

    const int64_t TS = (int64_t)gridDim.x * warps, t0 = min(p.T, (int64_t)blockIdx.x * warps + warp), t1 = p.T;
    const int items = t0 < t1 ? (int)((unsigned)(t1 - t0 + TS - 1) / (unsigned)TS) * p.parts : 0;  // this warp's stages: token i / parts, share i % parts
    const int row = p.d * (int)sizeof(T);
    // the heads [from, to) of job j in a share of the heads [ha, hb), at `src` of the stage
    struct Piece {
        int from, to;
        uint32_t src;
    };
    auto piece = [&](int j, int first, int ha, int hb) {
        const int from = max(ha, first), to = min(hb, first + p.jobs[j].heads);
        return Piece{from - first, to - first, (uint32_t)((from - ha) * row)};
    };
    auto share = [&](int part, int &ha, int &hb) {
        ha = part * p.share;
        hb = min(p.total_heads, ha + p.share);
    };
    // A walk over the items: stage, its use (odd or even), share and token, counted rather than divided.
    struct Item {
        int i, st, part;
        uint32_t use;
        int64_t t;
    };
    auto step = [&](Item &x) {
        ++x.i;
        if (++x.st == p.stages) {
            x.st = 0;
            x.use ^= 1u;
        }
        if (++x.part == p.parts) {
            x.part = 0;
            x.t += TS;
        }
    };
    Item ld{0, 0, 0, 0, t0};
    auto load = [&]() {  // lane 0: the next item
        int ha, hb;
        share(ld.part, ha, hb);
        uint8_t *dst = ring + ld.st * p.stage_bytes;
        uint64_t *bar = &full[warp][ld.st];
        dev::mbar_arrive_expect_tx(bar, (uint32_t)((hb - ha) * row));
        for (int j = 0, first = 0; j < p.njobs; first += p.jobs[j++].heads) {
            const Piece q = piece(j, first, ha, hb);
            if (q.from < q.to)
                dev::bulk_load(dst + q.src,
                               static_cast<const T *>(p.jobs[j].x) + ld.t * p.jobs[j].x_stride + (int64_t)q.from * p.d,
                               (uint32_t)((q.to - q.from) * row), bar);
        }
        step(ld);
    };
    if (lane == 0)
        while (ld.i < min(items, p.stages - 2)) load();
    const int hpi = 32 / p.rot_units, hh = lane / p.rot_units, u = lane % p.rot_units;
    const int off0 = u * 16, off1 = p.n_pairs * (int)sizeof(T) + u * 16, pb = u * NP;
    int rotated = 0;  // heads, which come first
    for (int j = 0; j < p.njobs; ++j) rotated += p.jobs[j].rotate ? p.jobs[j].heads : 0;
    // this lane's pairs: angle a position, and where its positions are
    unsigned long long turns[4];
    const int32_t *pos_at[4];
    int pos[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int w = min(lane + 32 * k, p.n_pairs - 1);
        turns[k] = p.turns[w];
        pos_at[k] = p.pos + (int64_t)p.axis[w] * p.T;
        pos[k] = t0 < t1 ? __ldg(pos_at[k] + t0) : 0;
    }
    // the sequence of the token in hand, its page, and the angles of this lane's unit
    int seq = -1, page = -1, page_i = -1, ok = 1;
    long long c0 = 0, c1 = -1, len = 0, off = 0;
    float rc[NP] = {}, rs[NP] = {};
    for (Item it{0, 0, 0, 0, t0}; it.i < items; step(it)) {
        const int64_t t = it.t;
        // the stores of the item before last have read their stage: it takes the next item
        dev::bulk_wait_read<1>();
        __syncwarp();
        if (lane == 0 && ld.i < items) load();
        // (the wait ahead of the angles, which paces the warps: 32768 tokens of 40 heads 105.4 us, behind them 109.6; 8192
        // of 72 heads 53.9 and 53.4, packed prefill appended 194.4 and 193.1)
        if (!dev::mbar_wait_warp(&full[warp][it.st], it.use, wc)) break;
        if (it.part == 0) {
            if (p.cu) {
                if (t >= c1) {
                    seq = dev::segment_of(p.cu + 1, p.B, t);
                    page_i = -1;
                    if (seq < p.B) {
                        c0 = p.cu[seq];
                        c1 = p.cu[seq + 1];
                        len = p.kv_lens[seq];
                    } else {
                        c1 = p.T;  // behind the last sequence, to the end
                    }
                }
                ok = 0;
                if (seq < p.B) {
                    const long long idx = len - (c1 - c0) + (t - c0);
                    bool in = t >= c0 && idx >= 0 && idx < p.table_keys;
                    if (in) {
                        const int pi = page_of(p, (int)idx);
                        if (pi != page_i) {
                            page_i = pi;
                            page = p.page_table[(int64_t)seq * p.table_width + pi];
                        }
                        in = page >= 0 && page < p.n_pages;
                        off = page * p.page_stride + ((int)idx - pi * p.page_size) * p.token_stride;
                    }
                    ok = in ? 2 : 1;
                    if (!in && lane == 0) dev::record_status(p.status, RA_ERR_DEVICE_BOUNDS);
                }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int w = lane + 32 * k;
                if (w < p.n_pairs) {
                    cs[w] = angle(pos[k], turns[k], p.inverse);
                    if (t + TS < t1) pos[k] = __ldg(pos_at[k] + t + TS);
                }
            }
            __syncwarp();
            if (hh < hpi) {
#pragma unroll
                for (int e = 0; e < NP; ++e) {
                    const float2 r = cs[pb + e];
                    rc[e] = r.x;
                    rs[e] = r.y;
                }
            }
        }
        int ha, hb;
        share(it.part, ha, hb);
        uint8_t *tok = ring + it.st * p.stage_bytes;
        if (hh < hpi) {
            const int most = min(hb, rotated) - ha;
#pragma unroll 4
            for (int h = hh; h < most; h += hpi) {
                V *pa = reinterpret_cast<V *>(tok + h * row + off0), *pb2 = reinterpret_cast<V *>(tok + h * row + off1);
                V a = *pa, b;
                if (!ADJ) b = *pb2;
                turn_unit<T, VEC, ADJ, NP>(a, b, rc, rs);
                *pa = a;
                if (!ADJ) *pb2 = b;
            }
        }
        dev::fence_proxy_async_smem();
        __syncwarp();
        for (int j = 0, first = 0; j < p.njobs; first += p.jobs[j++].heads) {
            const RopeJob &jb = p.jobs[j];
            const Piece q = piece(j, first, ha, hb);
            if (q.from >= q.to || ok < (jb.paged ? 2 : 1)) continue;
            T *y = static_cast<T *>(jb.y) + (jb.paged ? off + q.from * p.head_stride : t * jb.y_stride + (int64_t)q.from * p.d);
            if (!jb.paged || p.head_stride == p.d) {
                if (lane == 0) dev::bulk_store(y, tok + q.src, (uint32_t)((q.to - q.from) * row));
            } else {
                for (int h = lane; h < q.to - q.from; h += 32)
                    dev::bulk_store(y + h * p.head_stride, tok + q.src + h * row, (uint32_t)row);
            }
        }
        dev::bulk_commit();
    }
    // nothing may be under way when the CTA's shared memory goes
    dev::bulk_wait_all();
    if (lane == 0) {
        volatile int local_abort = 0;
        const dev::WaitCtl drain{&local_abort, p.status, p.budget_ns};
        for (int i = max(0, ld.i - p.stages); i < ld.i; ++i)
            (void)dev::mbar_wait(&full[warp][i % p.stages], (uint32_t)(i / p.stages) & 1u, drain);
    }
}

template <typename T>
cudaError_t launch_bulk(RopeParams &p, int sms, cudaStream_t st) {
    // four or more stages a warp, in kRingBytes
    // (with cache rows to find a warp waits longer between stages: smaller ones and more warps.  Stages of 5 and of
    // 8 KB: packed prefill appended 194 and 237 us; 32768 tokens rotated 105 and 105; 8192 of 72 heads 55.7 and 54.2)
    const int row = p.d * (int)sizeof(T), part = p.cu ? 5120 : 8192;
    p.parts = (p.total_heads * row + part - 1) / part;
    p.share = (p.total_heads + p.parts - 1) / p.parts;
    p.parts = (p.total_heads + p.share - 1) / p.share;
    p.stage_bytes = (p.share * row + 127) / 128 * 128;
    // (the angles of 128 pairs take some of the ring's room)
    const int fit = std::min(kRingBytes, kBulkSmem - kBulkWarps * p.n_pairs * (int)sizeof(float2)) / p.stage_bytes;
    const int warps = std::min(kBulkWarps, fit / 4);
    p.stages = std::min(kBulkStages, fit / warps);
    const int64_t blocks = std::min<int64_t>(sms, (p.T + warps - 1) / warps);
    const size_t smem = (size_t)warps * p.stages * p.stage_bytes + (size_t)warps * p.n_pairs * sizeof(float2);
    auto kernel = p.adjacent ? rope_bulk_kernel<T, true> : rope_bulk_kernel<T, false>;
    static LaunchFit half_split, adjacent;  // (the most that any call takes, so calls at once do not undo each other's)
    const cudaError_t e = (p.adjacent ? adjacent : half_split).prepare((const void *)kernel, warps * 32, kBulkSmem, nullptr);
    if (e != cudaSuccess) return e;
    kernel<<<(unsigned)blocks, warps * 32, smem, st>>>(p);
    return cudaGetLastError();
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
        // (of the magnitude, negated at the end: what a negative one lacks to a whole turn would lose its low bits)
        const double turns = std::fabs(inv_freq[i]) * 0.15915494309189533577;            // 1 / (2 pi)
        const double frac = turns - std::floor(turns);                                   // in [0, 1), exact
        const uint64_t part = (uint64_t)(frac * 18446744073709551616.0);                 // (exact: times 2^64)
        p.turns[i] = inv_freq[i] < 0 ? 0 - part : part;
        p.axis[i] = axes ? axes[i] : 0;
    }
}

cudaError_t launch_rope(RopeParams &p, int dtype, cudaStream_t st) {
    if (p.T <= 0) return cudaSuccess;
    p.status = device_status_ptr();
    p.budget_ns = wait_budget_ns();
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
    p.hpi = p.units > 32 ? 1 : 32 / p.units;
    p.unit_inv = (65535 + p.units) / p.units;
    for (int j = 0; j < p.njobs; ++j) p.jobs[j].groups = (p.jobs[j].heads + p.hpi - 1) / p.hpi;
    const int groups = (p.total_heads + p.hpi - 1) / p.hpi;
    // The ring kernel, which needs whole vectors and at most 32 units a head: for more tokens than the warp kernel
    // holds at once (20 warps an SM), and, rotating alone, for tokens of so many heads that the warps' loops over them
    // are longer.  (Heads of 128, warp kernel and ring.  40 heads: 3000 tokens 14.4 and 13.8 us, 3100 21.9 and 17.0,
    // 32768 140 and 104; 9 heads: 3000 tokens 7.2 and 9.5, 3500 10.8 and 9.5; 72 heads: 1000 tokens 9.9 and 9.3, 1400
    // 17.3 and 15.4, half of them rotated 29.6 and 12.6; 136 heads: 400 tokens 8.3 and 12.9, 1000 18.7 and 13.6.
    // Appended, 48 heads: 3000 tokens 17.8 and 19.3.)
    const int64_t sms = paged_sms();
    if (fast && p.n_pairs > 0 && p.rot_units <= 32 &&
        (p.T > kHeldWarps * sms || (!p.cu && p.T >= 4 * sms && p.T * groups > 144 * sms)))
        return dtype == RA_FP32 ? launch_bulk<float>(p, (int)sms, st) : launch_bulk<__nv_bfloat16>(p, (int)sms, st);
    // warps a token: enough to fill the GPU (16 warps an SM) when tokens are few, at most one per group of heads
    p.split = (int)std::min<int64_t>(groups, std::max<int64_t>(1, sms * 16 / p.T));
    if (dtype == RA_FP32) {
        if (!fast) return launch_warps<float, 1, false>(p, st);
        return adj ? launch_warps<float, 4, true>(p, st) : launch_warps<float, 4, false>(p, st);
    }
    if (!fast) return launch_warps<__nv_bfloat16, 1, false>(p, st);
    return adj ? launch_warps<__nv_bfloat16, 8, true>(p, st) : launch_warps<__nv_bfloat16, 8, false>(p, st);
}

}  // namespace ra

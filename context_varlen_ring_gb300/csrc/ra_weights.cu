// ra_weights.cu -- the attention weight that each cached key gathers from a
// batch's new tokens: w[key, KV head] += sum over the query rows that see the
// key of exp(scale q.k - lse), what eviction from the cache goes by.
//
// A unit is a tile of keys of one KV head: its CTA loads the keys once, walks
// the query rows that see them and owns their sums, so nothing is added by two
// CTAs and the order of the sums is fixed.  Scores have keys as rows and query
// rows as columns: a key's sum is then a sum over columns, which stays in the
// thread that has the key until the tile ends.  The units of all sequences and
// prefixes form one line, which the CTAs take in strides.
//
// Bound: with the few rows of a decoding step, memory (each key read once: 64
// sequences of up to 8192 keys, 8 heads, 51 us, 4.9 TB/s); with a chunk of
// hundreds of tokens, the products and exponentials; in fp32 the multiplications
// (9 sequences behind prefixes of up to 1500 keys, 16 us).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "ra_dev.cuh"
#include "ra_keep.h"
#include "ra_kernels.h"
#include "ra_serve.cuh"
#include "ra_weights.cuh"

namespace ra {
namespace {

using namespace dev;
using namespace weights;
using bf16 = __nv_bfloat16;

constexpr int kThreads = 128;
// ------------------------------------------------------------ bf16, warp-level products
__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int D, int KEYS>
struct MmaSmem {
    static constexpr int WK = KEYS / 16, WR = 4 / WK;  // warps along the keys, along the rows
    static constexpr int RB = 16 * WR < 32 ? 32 : 16 * WR;  // query rows a step
    static constexpr int LD = D + 8;
    bf16 k[KEYS][LD];
    bf16 q[2][RB][LD];
    float lse[2][RB];
    float sum[WR][KEYS];
    Line line;
};

template <int D, int KEYS>
__global__ void __launch_bounds__(kThreads) weights_mma_kernel(const WeightArgs a) {
    using Smem = MmaSmem<D, KEYS>;
    constexpr int WK = Smem::WK, WR = Smem::WR, RB = Smem::RB, RW = RB / WR;  // rows a step and warp
    constexpr int LOG = KEYS == 16 ? 4 : KEYS == 32 ? 5 : 6;
    extern __shared__ __align__(128) uint8_t raw[];
    Smem &sm = *reinterpret_cast<Smem *>(raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, wk = warp % WK, wr = warp / WK;
    const int S = a.B + a.n_groups;
    for (int s0 = S > kSegs ? 0 : -1; s0 >= 0 && s0 < S; s0 += kSegs)  // (nothing is added where any segment is bad)
        if (line_up<kThreads>(a, s0, LOG, sm.line) < 0) {
            if (tid == 0) record_status(a.status, RA_ERR_DEVICE_BOUNDS);
            return;
        }
    for (int s0 = 0; s0 < S; s0 += kSegs) {
        const int tiles = line_up<kThreads>(a, s0, LOG, sm.line);
        if (tiles < 0) {
            if (tid == 0) record_status(a.status, RA_ERR_DEVICE_BOUNDS);
            return;
        }
        for (int64_t u = blockIdx.x; u < (int64_t)tiles * a.Hkv; u += gridDim.x) {
            const int tile = (int)(u / a.Hkv), h = (int)(u - (int64_t)tile * a.Hkv);
            const int i = find(sm.line, tile), s = s0 + i, k0 = (tile - sm.line.at[i]) * KEYS;
            Segment g;
            segment(a, s, g);
            const bool own = s < a.B;
            const int rows = g.n * a.G;
            // the first row that sees a key of the tile
            const int first = own && a.causal ? max(0, k0 - (g.len - g.n)) * a.G : 0;
            __syncthreads();  // (the last unit's reads)
            for (int x = tid; x < KEYS * (D / 8); x += kThreads) {
                const int r = x / (D / 8), c = x % (D / 8) * 8;
                int64_t page = 0;
                int row = 0;
                const bool there = k0 + r < g.len && place(a, s, k0 + r, page, row);
                cp16(smem_u32(&sm.k[r][c]),
                     static_cast<const bf16 *>(a.k) + (there ? page * a.page_stride + row * a.token_stride + h * a.head_stride : 0) + c,
                     there);
            }
            auto load_q = [&](int r0, int buf) {
                for (int x = tid; x < RB * (D / 8); x += kThreads) {
                    const int r = r0 + x / (D / 8), c = x % (D / 8) * 8;
                    const bool there = r < rows;
                    const int t = token_of(a, there ? r : 0);
                    cp16(smem_u32(&sm.q[buf][x / (D / 8)][c]),
                         static_cast<const bf16 *>(a.q) + (g.tok0 + t) * a.q_stride + (h * a.G + (there ? r : 0) - t * a.G) * D + c,
                         there);
                }
                for (int x = tid; x < RB; x += kThreads) sm.lse[buf][x] = row_lse(a, g, h, r0 + x);
                asm volatile("cp.async.commit_group;" ::: "memory");
            };
            load_q(first, 0);
            float sum[2] = {0.f, 0.f};
            const int key = k0 + wk * 16 + (lane >> 2);  // and key + 8
            uint32_t fa[D / 16][4];
            for (int r0 = first, buf = 0; r0 < rows; r0 += RB, buf ^= 1) {
                if (r0 + RB < rows) {
                    load_q(r0 + RB, buf ^ 1);
                    asm volatile("cp.async.wait_group 1;" ::: "memory");
                } else {
                    asm volatile("cp.async.wait_group 0;" ::: "memory");
                }
                __syncthreads();
                if (r0 == first) {
                    const uint32_t ka = smem_u32(&sm.k[wk * 16 + (lane & 15)][(lane >> 4) * 8]);
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) ldsm4(ka + k * 32, fa[k]);
                }
                const bool masked = own && a.causal && g.len - g.n + token_of(a, r0) + 1 < k0 + KEYS;
#pragma unroll
                for (int n = 0; n < RW / 16; ++n) {
                    const int rw = wr * RW + n * 16;
                    float c0[4] = {0.f, 0.f, 0.f, 0.f}, c1[4] = {0.f, 0.f, 0.f, 0.f};
                    const uint32_t qa = smem_u32(&sm.q[buf][rw + (lane >> 4) * 8 + (lane & 7)][(lane >> 3 & 1) * 8]);
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        uint32_t fb[4];
                        ldsm4(qa + k * 32, fb);
                        mma16816(c0, fa[k], fb[0], fb[1]);
                        mma16816(c1, fa[k], fb[2], fb[3]);
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) {  // columns rw + 2 (lane % 4) + {0, 1, 8, 9}
                        const int col = rw + 2 * (lane & 3) + (e & 1) + (e >> 1) * 8;
                        const float off = sm.lse[buf][col];
                        const float *c = e >> 1 ? c1 : c0;
                        float p0 = ex2_approx(fmaf(c[e & 1], a.scale_log2, off));
                        float p1 = ex2_approx(fmaf(c[2 + (e & 1)], a.scale_log2, off));
                        if (off == -INFINITY) p0 = p1 = 0.f;  // (a padded or empty row adds nothing, whatever the key)
                        if (masked) {
                            const int limit = limit_of(a, g, true, r0 + col);
                            if (key >= limit) p0 = 0.f;
                            if (key + 8 >= limit) p1 = 0.f;
                        }
                        sum[0] += p0;
                        sum[1] += p1;
                    }
                }
                __syncthreads();
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], 1);
                sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], 2);
                if ((lane & 3) == 0) sm.sum[wr][wk * 16 + (lane >> 2) + 8 * e] = sum[e];
            }
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            __syncthreads();
            for (int r = tid; r < KEYS; r += kThreads) {
                int64_t page;
                int row;
                if (k0 + r >= g.len || !place(a, s, k0 + r, page, row)) continue;
                float x = 0.f;
#pragma unroll
                for (int w = 0; w < WR; ++w) x += sm.sum[w][r];
                a.w[page * a.w_page + row * a.w_token + h * a.w_head] += x;
            }
        }
    }
}

// ------------------------------------------------------------ bf16, few query rows: a stream of keys a warp
// A decoding step has G rows a KV head, one 16-row block of products for each 16 keys, and reads 2 D bytes a key.  Every
// warp streams its own runs of keys through a private ring of kRing blocks of 16; a block's keys and old weights come by
// asynchronous copies, its page is looked up a block ahead of them, and the rows stay in registers.  More rows are taken
// block by block against each 16 keys.  A warp's blocks are one piece of the line of all segments' heads, so that it
// searches for a segment, and loads its rows, once or twice (64 sequences of up to 8192 keys, in runs of 64 or 256 keys
// dealt out to the warps in turn: 67 us, so 54; with one address a lane, 51).
constexpr int kRing = 3, kStreamWarps = 16, kStreamThreads = 32 * kStreamWarps;

template <int D>
struct StreamSmem {
    uint8_t k[kStreamWarps][kRing][16 * D * 2];
    float old[kStreamWarps][kRing][16];
    int64_t w[kStreamWarps][kRing][16];  // where the weights are; -1: none
    Line line;
};

template <int D>
__global__ void __launch_bounds__(kStreamThreads) weights_stream_kernel(const WeightArgs a) {
    constexpr int CPR = D / 8, RPI = 32 / CPR;  // 16-byte pieces a row, rows a warp instruction
    extern __shared__ __align__(128) uint8_t raw[];
    StreamSmem<D> &sm = *reinterpret_cast<StreamSmem<D> *>(raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int S = a.B + a.n_groups;
    for (int s0 = S > kSegs ? 0 : -1; s0 >= 0 && s0 < S; s0 += kSegs)
        if (line_up<kStreamThreads>(a, s0, 4, sm.line) < 0) {
            if (tid == 0) record_status(a.status, RA_ERR_DEVICE_BOUNDS);
            return;
        }
    const uint32_t ring = smem_u32(sm.k[warp]), olds = smem_u32(sm.old[warp]);
    const int64_t warps = (int64_t)gridDim.x * kStreamWarps, self = (int64_t)blockIdx.x * kStreamWarps + warp;
    for (int s0 = 0; s0 < S; s0 += kSegs) {
        const int tiles = line_up<kStreamThreads>(a, s0, 4, sm.line);
        if (tiles < 0) {
            if (tid == 0) record_status(a.status, RA_ERR_DEVICE_BOUNDS);
            return;
        }
        // this warp's blocks of 16 keys: an equal share of all (segment, head, block), one behind the other
        struct Place {
            int64_t u;  // the block
            int s, h, k, len;
        };
        const int64_t blocks = (int64_t)tiles * a.Hkv, share = blocks / warps, rest = blocks % warps;
        const int64_t u0 = self * share + min(self, rest), u1 = u0 + share + (self < rest);
        auto enter = [&](Place &p) {  // the block's segment; false behind the last
            if (p.u >= u1) return false;
            const int i = find(sm.line, (int)(p.u / a.Hkv));
            const int64_t off = p.u - (int64_t)sm.line.at[i] * a.Hkv;
            const int n = sm.line.at[i + 1] - sm.line.at[i];
            Segment g;
            p.h = (int)(off / n);
            p.s = s0 + i;
            p.k = (int)(off - (int64_t)p.h * n) * 16;
            segment(a, p.s, g);
            p.len = g.len;
            return true;
        };
        auto advance = [&](Place &p) {
            if (++p.u >= u1) return false;
            p.k += 16;
            if (p.k < p.len) return true;
            p.k = 0;
            return ++p.h < a.Hkv || enter(p);
        };
        const bool whole = a.page_shift >= 4;  // a block is on one page
        // the page of this lane's key of a block (lanes 0 .. 15), as the table has it
        auto look_up = [&](const Place &p) {
            const int f = p.s >= a.B, i = p.s - (f ? a.B : 0), key = p.k + (whole ? 0 : lane & 15);
            const int pi = a.page_shift >= 0 ? key >> a.page_shift : key / a.page_size;
            return key < p.len ? __ldg(a.table[f] + (int64_t)i * a.width[f] + pi) : -1;
        };
        int head = 0, tail = 0;
        auto load = [&](const Place &p, int page) {
            if (whole) {  // (one address a lane, and no exchange of them: 53.8 -> 51.9 us)
                const int row = p.k & (a.page_size - 1), n = p.len - p.k;
                const bool there = page >= 0 && page < a.n_pages;
                if (!there) record_status(a.status, RA_ERR_DEVICE_BOUNDS);
                if (lane < 16) {
                    const bool mine = there && lane < n;
                    const int64_t w = page * a.w_page + (row + lane) * a.w_token + p.h * a.w_head;
                    sm.w[warp][head][lane] = mine ? w : -1;
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(olds + (head * 16 + lane) * 4),
                                 "l"(a.w + (mine ? w : 0)), "r"(mine ? 4 : 0)
                                 : "memory");
                }
                const int c = lane % CPR, r0 = lane / CPR;
                const uint32_t dst = ring + head * (16 * D * 2);
                const int64_t o = there ? page * a.page_stride + (row + r0) * a.token_stride + p.h * a.head_stride : 0;
                const bf16 *src = static_cast<const bf16 *>(a.k) + o + c * 8;
#pragma unroll
                for (int i = 0; i < 16 / RPI; ++i) {
                    const int r = i * RPI + r0;
                    const bool mine = there && r < n;
                    cp16(dst + r * (D * 2) + ((c ^ (r & 7)) << 4), mine ? src : static_cast<const bf16 *>(a.k), mine);
                    src += RPI * a.token_stride;
                }
                head = head + 1 == kRing ? 0 : head + 1;
                return;
            }
            const int key = p.k + (lane & 15), pi = a.page_shift >= 0 ? key >> a.page_shift : key / a.page_size;
            const int row = key - pi * a.page_size;
            const bool there = key < p.len && page >= 0 && page < a.n_pages;
            if (key < p.len && !there) record_status(a.status, RA_ERR_DEVICE_BOUNDS);
            const int64_t off = there ? page * a.page_stride + row * a.token_stride + p.h * a.head_stride : -1;
            const int64_t w = there ? page * a.w_page + row * a.w_token + p.h * a.w_head : -1;
            if (lane < 16) {
                sm.w[warp][head][lane] = w;
                asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(olds + (head * 16 + lane) * 4),
                             "l"(a.w + (there ? w : 0)), "r"(there ? 4 : 0)
                             : "memory");
            }
            const int c = lane % CPR, r0 = lane / CPR;
            const uint32_t dst = ring + head * (16 * D * 2);
#pragma unroll
            for (int i = 0; i < 16 / RPI; ++i) {
                const int r = i * RPI + r0;
                const int64_t o = __shfl_sync(0xffffffffu, off, r);
                cp16(dst + r * (D * 2) + ((c ^ (r & 7)) << 4), static_cast<const bf16 *>(a.k) + (o < 0 ? 0 : o) + c * 8, o >= 0);
            }
            head = head + 1 == kRing ? 0 : head + 1;
        };
        Place in, at;
        in.u = u0;
        bool more = enter(in);
        at = in;
        bool left = more;
        int page = more ? look_up(in) : -1;
#pragma unroll 1
        for (int i = 0; i < kRing - 1; ++i) {
            if (more) {
                const Place now = in;
                const int p = page;
                more = advance(in);
                if (more) page = look_up(in);
                load(now, p);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
        int64_t held = -1;  // the segment and head whose rows are in registers
        uint32_t fb[D / 16][4];
        float off[4];
        Segment g{};
        int rows = 0;
        // rows r0 .. r0 + 15 as the products' columns, straight from the tensor: 4 bytes a place
        auto rows_of = [&](int h, int r0) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = r0 + 8 * e + (lane >> 2);
                const bool there = r < rows;
                const int t = token_of(a, there ? r : 0);
                const bf16 *q = static_cast<const bf16 *>(a.q) + (g.tok0 + t) * a.q_stride + (h * a.G + (there ? r : 0) - t * a.G) * D + 2 * (lane & 3);
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    fb[k][2 * e] = there ? __ldg(reinterpret_cast<const uint32_t *>(q + 16 * k)) : 0u;
                    fb[k][2 * e + 1] = there ? __ldg(reinterpret_cast<const uint32_t *>(q + 16 * k + 8)) : 0u;
                }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) off[e] = row_lse(a, g, h, r0 + 2 * (lane & 3) + (e & 1) + (e >> 1) * 8);
        };
        while (left) {
            const int k0 = at.k;
            const bool own = at.s < a.B;
            const int64_t want = (int64_t)at.s * a.Hkv + at.h;
            if (want != held) {
                segment(a, at.s, g);
                rows = g.n * a.G;
            }
            const int first = own && a.causal ? max(0, k0 - (g.len - g.n)) * a.G & ~15 : 0;
            if (want != held && rows <= 16) rows_of(at.h, 0);
            held = want;
            asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 2) : "memory");
            __syncwarp();
            uint32_t fa[D / 16][4];
            const uint32_t ka = ring + tail * (16 * D * 2) + (lane & 15) * (D * 2);
#pragma unroll
            for (int k = 0; k < D / 16; ++k) ldsm4(ka + (((2 * k + (lane >> 4)) ^ (lane & 7)) << 4), fa[k]);
            const int mine = (lane >> 2) + 8 * (lane & 1);  // the key that this lane writes (lanes 0 and 1 of each four)
            const float old = sm.old[warp][tail][mine];
            const int64_t w = sm.w[warp][tail][mine];
            tail = tail + 1 == kRing ? 0 : tail + 1;
            __syncwarp();  // (the block can be loaded over)
            if (more) {
                const Place now = in;
                const int p = page;
                more = advance(in);
                if (more) page = look_up(in);
                load(now, p);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
            float sum[2] = {0.f, 0.f};
            const int key = k0 + (lane >> 2);
            for (int r0 = first; r0 < rows; r0 += 16) {
                if (rows > 16) rows_of(at.h, r0);
                float c[2][4] = {}, c2[4] = {};
                const bool both = r0 + 8 < rows;  // rows in the second half of the block
#pragma unroll
                for (int k = 0; k < D / 16; k += 2) {  // (two chains of products)
                    mma16816(c[0], fa[k], fb[k][0], fb[k][1]);
                    mma16816(c2, fa[k + 1], fb[k + 1][0], fb[k + 1][1]);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) c[0][e] += c2[e];
                if (both) {
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) mma16816(c[1], fa[k], fb[k][2], fb[k][3]);
                }
                const bool masked = own && a.causal && g.len - g.n + token_of(a, r0) + 1 < k0 + 16;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (e >= 2 && !both) break;
                    const float *x = c[e >> 1];
                    float p0 = ex2_approx(fmaf(x[e & 1], a.scale_log2, off[e]));
                    float p1 = ex2_approx(fmaf(x[2 + (e & 1)], a.scale_log2, off[e]));
                    if (off[e] == -INFINITY) p0 = p1 = 0.f;
                    if (masked) {
                        const int limit = limit_of(a, g, true, r0 + 2 * (lane & 3) + (e & 1) + (e >> 1) * 8);
                        if (key >= limit) p0 = 0.f;
                        if (key + 8 >= limit) p1 = 0.f;
                    }
                    sum[0] += p0;
                    sum[1] += p1;
                }
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], 1);
                sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], 2);
            }
            if ((lane & 3) < 2 && w >= 0) a.w[w] = old + sum[lane & 1];
            left = advance(at);
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();
    }
}

// ------------------------------------------------------------ fp32 arithmetic: fp32, and bf16 of other head sizes
// 32 keys by 64 rows a step; the next step's rows are on their way to registers beside it (9 sequences of a few tokens
// behind prefixes of 1500 keys, heads of 64: 31 us with 32 rows a step, loaded when due, 17 so).
constexpr int kSimtKeys = 32, kSimtRows = 64, kSimtThreads = 256;

struct SimtSmem {
    float lse[kSimtRows];
    float sum[16][kSimtKeys];
    Line line;
};

// P: pieces of 4 elements that a thread loads of a row, four threads a row (d <= 16 P).
template <typename E, int P>
__global__ void __launch_bounds__(kSimtThreads) weights_simt_kernel(const WeightArgs a) {
    extern __shared__ __align__(128) uint8_t raw[];
    SimtSmem &sm = *reinterpret_cast<SimtSmem *>(raw);
    const int ld = a.d + 4;
    float *sk = reinterpret_cast<float *>(raw + (sizeof(SimtSmem) + 127) / 128 * 128), *sq = sk + kSimtKeys * ld;
    const int tid = threadIdx.x, kx = tid & 15, ry = tid >> 4;
    const int S = a.B + a.n_groups;
    for (int s0 = S > kSegs ? 0 : -1; s0 >= 0 && s0 < S; s0 += kSegs)
        if (line_up<kSimtThreads>(a, s0, 5, sm.line) < 0) {
            if (tid == 0) record_status(a.status, RA_ERR_DEVICE_BOUNDS);
            return;
        }
    auto get4 = [&](const E *src, bool there) {
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (there) {
            if (sizeof(E) == 4) {
                x = *reinterpret_cast<const float4 *>(src);
            } else {
                const uint2 y = *reinterpret_cast<const uint2 *>(src);
                const float2 p = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&y.x));
                const float2 r = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&y.y));
                x = make_float4(p.x, p.y, r.x, r.y);
            }
        }
        return x;
    };
    const int vec = a.d / 4;
    for (int s0 = 0; s0 < S; s0 += kSegs) {
        const int tiles = line_up<kSimtThreads>(a, s0, 5, sm.line);
        if (tiles < 0) {
            if (tid == 0) record_status(a.status, RA_ERR_DEVICE_BOUNDS);
            return;
        }
        for (int64_t u = blockIdx.x; u < (int64_t)tiles * a.Hkv; u += gridDim.x) {
            const int tile = (int)(u / a.Hkv), h = (int)(u - (int64_t)tile * a.Hkv);
            const int i = find(sm.line, tile), s = s0 + i, k0 = (tile - sm.line.at[i]) * kSimtKeys;
            Segment g;
            segment(a, s, g);
            const bool own = s < a.B;
            const int rows = g.n * a.G;
            const int first = own && a.causal ? max(0, k0 - (g.len - g.n)) * a.G : 0;
            // rows r0 .. of q: this thread's row and pieces, and the row's offset
            float4 next[P];
            float next_lse = 0.f;
            auto look = [&](int r0) {
                const int r = r0 + (tid >> 2);
                const bool there = r < rows;
                const int t = token_of(a, there ? r : 0);
                const E *q = static_cast<const E *>(a.q) + (g.tok0 + t) * a.q_stride + (int64_t)(h * a.G + (there ? r : 0) - t * a.G) * a.d;
#pragma unroll
                for (int e = 0; e < P; ++e) {
                    const int c = (tid & 3) + 4 * e;
                    next[e] = get4(q + c * 4, there && c < vec);
                }
                if (tid < kSimtRows) next_lse = row_lse(a, g, h, r0 + tid);
            };
            look(first);
            __syncthreads();  // (the last unit's reads)
            {
                const int r = tid >> 3;
                int64_t page = 0;
                int row = 0;
                const bool there = k0 + r < g.len && place(a, s, k0 + r, page, row);
                const E *k = static_cast<const E *>(a.k) + (there ? page * a.page_stride + row * a.token_stride + h * a.head_stride : 0);
                for (int c = tid & 7; c < vec; c += 8) *reinterpret_cast<float4 *>(sk + r * ld + c * 4) = get4(k + c * 4, there);
            }
            float sum[2] = {0.f, 0.f};
            for (int r0 = first; r0 < rows; r0 += kSimtRows) {
                __syncthreads();
#pragma unroll
                for (int e = 0; e < P; ++e) {
                    const int c = (tid & 3) + 4 * e;
                    if (c < vec) *reinterpret_cast<float4 *>(sq + (tid >> 2) * ld + c * 4) = next[e];
                }
                if (tid < kSimtRows) sm.lse[tid] = next_lse;
                __syncthreads();
                if (r0 + kSimtRows < rows) look(r0 + kSimtRows);
                float acc[2][4] = {};
#pragma unroll 4
                for (int c = 0; c < a.d; c += 4) {
                    float4 k[2], q[4];
#pragma unroll
                    for (int e = 0; e < 2; ++e) k[e] = *reinterpret_cast<const float4 *>(sk + (kx + 16 * e) * ld + c);
#pragma unroll
                    for (int e = 0; e < 4; ++e) q[e] = *reinterpret_cast<const float4 *>(sq + (ry + 16 * e) * ld + c);
#pragma unroll
                    for (int e = 0; e < 2; ++e)
#pragma unroll
                        for (int f = 0; f < 4; ++f)
                            acc[e][f] += k[e].x * q[f].x + k[e].y * q[f].y + k[e].z * q[f].z + k[e].w * q[f].w;
                }
#pragma unroll
                for (int f = 0; f < 4; ++f) {
                    const int row = ry + 16 * f;
                    const float off = sm.lse[row];
                    if (off == -INFINITY) continue;
                    const int limit = limit_of(a, g, own, r0 + row);
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        if (k0 + kx + 16 * e < limit) sum[e] += exp2f(fmaf(acc[e][f], a.scale_log2, off));
                }
            }
            sm.sum[ry][kx] = sum[0];
            sm.sum[ry][kx + 16] = sum[1];
            __syncthreads();
            if (tid < kSimtKeys) {
                int64_t page;
                int row;
                if (k0 + tid < g.len && place(a, s, k0 + tid, page, row)) {
                    float x = 0.f;
#pragma unroll
                    for (int w = 0; w < 16; ++w) x += sm.sum[w][tid];
                    a.w[page * a.w_page + row * a.w_token + h * a.w_head] += x;
                }
            }
        }
    }
}

template <typename E, int P>
cudaError_t simt_launch(const WeightArgs &a, cudaStream_t st) {
    static LaunchFit fit;
    auto kernel = weights_simt_kernel<E, P>;
    const size_t fixed = (sizeof(SimtSmem) + 127) / 128 * 128;
    int ctas = 0;  // (of the largest heads)
    const cudaError_t e = fit.prepare(reinterpret_cast<const void *>(kernel), kSimtThreads,
                                      fixed + (kSimtKeys + kSimtRows) * (16 * P + 4) * 4, &ctas);
    if (e != cudaSuccess) return e;
    kernel<<<paged_sms() * ctas, kSimtThreads, fixed + (size_t)(kSimtKeys + kSimtRows) * (a.d + 4) * 4, st>>>(a);
    return cudaGetLastError();
}

template <int D, int KEYS>
cudaError_t mma_launch(const WeightArgs &a, cudaStream_t st) {
    static LaunchFit fit;
    auto kernel = weights_mma_kernel<D, KEYS>;
    int ctas = 0;
    const cudaError_t e = fit.prepare(reinterpret_cast<const void *>(kernel), kThreads, sizeof(MmaSmem<D, KEYS>), &ctas);
    if (e != cudaSuccess) return e;
    kernel<<<paged_sms() * ctas, kThreads, sizeof(MmaSmem<D, KEYS>), st>>>(a);
    return cudaGetLastError();
}
template <int D>
cudaError_t mma_keys(const WeightArgs &a, int keys, cudaStream_t st) {
    return keys == 16 ? mma_launch<D, 16>(a, st) : keys == 32 ? mma_launch<D, 32>(a, st) : mma_launch<D, 64>(a, st);
}

template <int D>
cudaError_t stream_launch(const WeightArgs &a, cudaStream_t st) {
    static LaunchFit fit;
    auto kernel = weights_stream_kernel<D>;
    int ctas = 0;
    const cudaError_t e = fit.prepare(reinterpret_cast<const void *>(kernel), kStreamThreads, sizeof(StreamSmem<D>), &ctas);
    if (e != cudaSuccess) return e;
    kernel<<<paged_sms() * ctas, kStreamThreads, sizeof(StreamSmem<D>), st>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_weights_stream(const WeightArgs &a, cudaStream_t st) {
    return a.d == 64 ? stream_launch<64>(a, st) : stream_launch<128>(a, st);
}
bool weights_mma_supported(int dtype, int d) { return dtype == RA_BF16 && (d == 64 || d == 128); }
cudaError_t launch_weights_mma(const WeightArgs &a, int keys, cudaStream_t st) {
    return a.d == 64 ? mma_keys<64>(a, keys, st) : mma_keys<128>(a, keys, st);
}
cudaError_t launch_weights_simt(const WeightArgs &a, cudaStream_t st) {
    if (a.dtype == RA_FP32)
        return a.d <= 64 ? simt_launch<float, 4>(a, st) : a.d <= 128 ? simt_launch<float, 8>(a, st) : simt_launch<float, 16>(a, st);
    return a.d <= 64 ? simt_launch<bf16, 4>(a, st) : a.d <= 128 ? simt_launch<bf16, 8>(a, st) : simt_launch<bf16, 16>(a, st);
}

}  // namespace ra

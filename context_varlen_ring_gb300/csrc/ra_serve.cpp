// ra_serve.cpp -- the C entries of rotary positions, the paged-cache append
// and paged attention: argument checks, workspace layout and the choice of
// kernels.  Host code only.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <string>

#include "ra_internal.h"
#include "ra_kernels.h"

namespace ra {
namespace {

ra_status launch_failed(cudaError_t e, const char *what) {
    return fail(RA_ERR_CUDA, std::string(what) + ": " + cudaGetErrorString(e));
}

bool on16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
int elem(int dtype) { return dtype == RA_FP32 ? 4 : 2; }
bool on_elem(const void *p, int dtype) { return reinterpret_cast<uintptr_t>(p) % elem(dtype) == 0; }

int log2_or_none(int x) {
    for (int i = 0; i < 31; ++i)
        if (x == 1 << i) return i;
    return -1;
}

ra_status check_rope(const ra_rope *r, const int32_t *pos, int d) {
    if (!r->inv_freq || !pos) return fail(RA_ERR_INVALID_ARG, "inv_freq or pos is NULL");
    if (r->n_axes < 1 || r->n_axes > 8) return fail(RA_ERR_INVALID_ARG, "n_axes must be in [1, 8]");
    if (r->n_pairs < 1 || 2 * (int64_t)r->n_pairs > d)
        return fail(RA_ERR_INVALID_ARG, "n_pairs must be at least 1 and 2 * n_pairs at most d");
    for (int i = 0; i < r->n_pairs; ++i) {
        if (!std::isfinite(r->inv_freq[i])) return fail(RA_ERR_INVALID_ARG, "inv_freq must be finite");
        if (r->axes && r->axes[i] >= r->n_axes) return fail(RA_ERR_INVALID_ARG, "an axis lies outside [0, n_axes)");
    }
    return RA_OK;
}

ra_status check_rows(int dtype, int64_t T, int d) {
    if (dtype != RA_BF16 && dtype != RA_FP32) return fail(RA_ERR_INVALID_ARG, "dtype must be RA_BF16 or RA_FP32");
    if (T < 0 || T > INT32_MAX) return fail(RA_ERR_INVALID_ARG, "T must be in [0, 2^31)");
    if (d <= 0) return fail(RA_ERR_INVALID_ARG, "d must be positive");
    if (d % 4 != 0 || d > 256) return fail(RA_ERR_UNSUPPORTED, "d must be a multiple of 4 and <= 256");
    return RA_OK;
}

// Rows of H * d contiguous elements, `stride` apart.
ra_status check_tensor(const void *x, const void *y, int dtype, int H, int d, int64_t xs, int64_t ys,
                       const char *name) {
    if (H <= 0 || H > 4096) return fail(RA_ERR_INVALID_ARG, std::string("bad head count of ") + name);
    if (!x || !y) return fail(RA_ERR_INVALID_ARG, std::string(name) + " is NULL");
    if (xs < (int64_t)H * d || ys < (int64_t)H * d)
        return fail(RA_ERR_INVALID_ARG, std::string("row stride of ") + name + " is smaller than its heads");
    if (!on_elem(x, dtype) || !on_elem(y, dtype))
        return fail(RA_ERR_UNSUPPORTED, std::string(name) + " is not aligned to its elements");
    if (x == y && xs != ys)
        return fail(RA_ERR_INVALID_ARG, std::string(name) + ": an output on its input needs the input's stride");
    return RA_OK;
}

ra_status rope_common(const void *q, const void *k, void *qo, void *ko, int dtype, int64_t T, int Hq, int Hk, int d,
                      int64_t qs, int64_t ks, int64_t qos, int64_t kos, const int32_t *pos, const ra_rope *rope,
                      int inverse, void *stream) {
    ra_status st = check_rows(dtype, T, d);
    if (st) return st;
    if (!rope) return fail(RA_ERR_INVALID_ARG, "rope is NULL");
    if (T == 0) return RA_OK;
    if ((st = check_rope(rope, pos, d))) return st;
    if ((st = check_tensor(q, qo, dtype, Hq, d, qs, qos, "q"))) return st;
    if ((k == nullptr) != (ko == nullptr)) return fail(RA_ERR_INVALID_ARG, "k and k_out go together");
    if (k && (st = check_tensor(k, ko, dtype, Hk, d, ks, kos, "k"))) return st;
    RopeParams p{};
    p.jobs[p.njobs++] = RopeJob{q, qo, qs, qos, Hq, 1, 0};
    if (k) p.jobs[p.njobs++] = RopeJob{k, ko, ks, kos, Hk, 1, 0};
    p.d = d;
    p.T = T;
    p.pos = pos;
    rope_table(p, rope->inv_freq, rope->axes, rope->n_pairs, rope->adjacent, inverse);
    ProfScope ps(inverse ? "ra_rope_bwd" : "ra_rope_fwd", static_cast<cudaStream_t>(stream));
    const cudaError_t e = launch_rope(p, dtype, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? RA_OK : launch_failed(e, "rope launch");
}

ra_status check_cache(const ra_paged_kv *c) {
    if (!c) return fail(RA_ERR_INVALID_ARG, "cache is NULL");
    if (c->dtype != RA_BF16 && c->dtype != RA_FP32)
        return fail(RA_ERR_INVALID_ARG, "the cache's dtype must be RA_BF16 or RA_FP32");
    if (c->n_pages < 0 || c->n_pages > INT32_MAX || c->page_size < 1 || c->Hkv < 1 || c->Hkv > 4096 || c->d < 1)
        return fail(RA_ERR_INVALID_ARG, "bad cache shape");
    if (c->page_stride < 0 || c->token_stride < 0 || c->head_stride < 0)
        return fail(RA_ERR_INVALID_ARG, "the cache's strides must not be negative");
    return RA_OK;
}

// ------------------------------------------------------------ paged attention
// Where everything lies in the workspace.  The sizes hold for every kernel
// that a call of these shapes may choose (the choice also goes by the page
// size and the scale, which the size query does not know).
struct PagedLayout {
    size_t o_hdr[2], o_seg[2], o_start[2], o_acc[2], o_ml[2], bytes;
};

// The most query rows that a segment of the family has per KV head (as far as the hint goes).
int64_t paged_rows(int family, int64_t T, int G, int max_q_len) {
    return (family || max_q_len <= 0 ? T : std::min<int64_t>(max_q_len, T)) * G;
}

PagedLayout paged_layout(int64_t T, int B, int n_groups, int G, int Hkv, int d, int dtype, int max_q_len) {
    PagedLayout L{};
    size_t at = 0;
    auto take = [&](size_t n) {
        const size_t o = at;
        at = align_up(at + n, 256);
        return o;
    };
    for (int f = 0; f < 2; ++f) {
        const int64_t S = f ? n_groups : B;
        L.o_hdr[f] = take(sizeof(PagedHdr));
        L.o_seg[f] = take((size_t)S * sizeof(PagedSeg));
        L.o_start[f] = take((size_t)kPagedMaxCtas * 4);
        // the rows themselves (twice where units are halved), and one unit more a CTA
        const int64_t most = paged_rows(f, T, G, max_q_len);
        const bool wide = most > (f ? 16 : 32) && dtype == RA_BF16 && d == 128;
        int64_t rows = S ? T * G * Hkv + (int64_t)kPagedMaxCtas * (most <= 16 ? 16 : 64) : 0;
        if (S && wide) rows = std::max(rows, 2 * T * G * Hkv + (int64_t)kPagedMaxWide * kPagedWideRows);
        L.o_acc[f] = take((size_t)rows * d * 4);
        L.o_ml[f] = take((size_t)rows * 8);
    }
    L.bytes = at;
    return L;
}

ra_status check_paged_shape(int64_t T, int B, int n_groups, int Hq, int Hkv, int d, int dtype) {
    if (dtype != RA_BF16 && dtype != RA_FP32) return fail(RA_ERR_INVALID_ARG, "dtype must be RA_BF16 or RA_FP32");
    if (T < 0 || n_groups < 0 || B < 0 || (B == 0 && T > 0))
        return fail(RA_ERR_INVALID_ARG, "T and n_groups must be >= 0, B >= 1 (0 with T = 0: an empty batch)");
    if (Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0) return fail(RA_ERR_INVALID_ARG, "Hq must be a positive multiple of Hkv");
    if (d <= 0) return fail(RA_ERR_INVALID_ARG, "d must be positive");
    if (d % 32 != 0 || d > 256) return fail(RA_ERR_UNSUPPORTED, "d must be a multiple of 32 and <= 256");
    if (T > (1 << 30) / Hq) return fail(RA_ERR_UNSUPPORTED, "T * Hq must be at most 2^30");
    if (B > (1 << 20) || n_groups > (1 << 20) || (int64_t)Hkv * ((int64_t)B + n_groups) > (1 << 28))
        return fail(RA_ERR_UNSUPPORTED, "too many sequences");
    return RA_OK;
}

}  // namespace
}  // namespace ra

using namespace ra;

extern "C" {

ra_status ra_rope_fwd(const void *q, const void *k, void *q_out, void *k_out, int dtype, int64_t T, int Hq, int Hk,
                      int d, int64_t q_stride, int64_t k_stride, int64_t q_out_stride, int64_t k_out_stride,
                      const int32_t *pos, const ra_rope *rope, void *stream) {
    return rope_common(q, k, q_out, k_out, dtype, T, Hq, Hk, d, q_stride, k_stride, q_out_stride, k_out_stride, pos,
                       rope, 0, stream);
}

ra_status ra_rope_bwd(const void *dq, const void *dk, void *dq_out, void *dk_out, int dtype, int64_t T, int Hq,
                      int Hk, int d, int64_t dq_stride, int64_t dk_stride, int64_t dq_out_stride,
                      int64_t dk_out_stride, const int32_t *pos, const ra_rope *rope, void *stream) {
    return rope_common(dq, dk, dq_out, dk_out, dtype, T, Hq, Hk, d, dq_stride, dk_stride, dq_out_stride,
                       dk_out_stride, pos, rope, 1, stream);
}

ra_status ra_kv_cache_append(const void *k, const void *v, int64_t k_stride, int64_t v_stride, int64_t T,
                             const ra_paged_kv *cache, const int32_t *page_table, int64_t table_width,
                             const int32_t *cu_seqlens, const int32_t *kv_lens, int B, const void *q, void *q_out,
                             int Hq, int64_t q_stride, int64_t q_out_stride, const int32_t *pos, const ra_rope *rope,
                             void *stream) {
    ra_status st = check_cache(cache);
    if (st) return st;
    if ((st = check_rows(cache->dtype, T, cache->d))) return st;
    if (B < 0 || (B == 0 && T > 0) || table_width < 0 || table_width > INT32_MAX)
        return fail(RA_ERR_INVALID_ARG, "B must be >= 1 (0 with T = 0: an empty batch) and table_width in [0, 2^31)");
    if ((q == nullptr) != (q_out == nullptr)) return fail(RA_ERR_INVALID_ARG, "q and q_out go together");
    if (q && !rope) return fail(RA_ERR_INVALID_ARG, "queries are taken along to be rotated: q without rope");
    if (T == 0) return RA_OK;
    if (!cu_seqlens || !kv_lens || (table_width > 0 && !page_table))
        return fail(RA_ERR_INVALID_ARG, "a segment array is NULL");
    const int d = cache->d, dt = cache->dtype;
    if (!cache->k || !cache->v) return fail(RA_ERR_INVALID_ARG, "a cache is NULL");
    if (!on_elem(cache->k, dt) || !on_elem(cache->v, dt))
        return fail(RA_ERR_UNSUPPORTED, "a cache is not aligned to its elements");
    if ((st = check_tensor(k, cache->k, dt, cache->Hkv, d, k_stride, (int64_t)cache->Hkv * d, "k"))) return st;
    if ((st = check_tensor(v, cache->v, dt, cache->Hkv, d, v_stride, (int64_t)cache->Hkv * d, "v"))) return st;
    if (q && (st = check_tensor(q, q_out, dt, Hq, d, q_stride, q_out_stride, "q"))) return st;
    if (rope && (st = check_rope(rope, pos, d))) return st;
    RopeParams p{};
    if (q) p.jobs[p.njobs++] = RopeJob{q, q_out, q_stride, q_out_stride, Hq, 1, 0};
    p.jobs[p.njobs++] = RopeJob{k, cache->k, k_stride, 0, cache->Hkv, rope ? 1 : 0, 1};
    p.jobs[p.njobs++] = RopeJob{v, cache->v, v_stride, 0, cache->Hkv, 0, 1};
    p.d = d;
    p.T = T;
    p.pos = pos;
    if (rope) rope_table(p, rope->inv_freq, rope->axes, rope->n_pairs, rope->adjacent, 0);
    p.cu = cu_seqlens;
    p.kv_lens = kv_lens;
    p.page_table = page_table;
    p.table_width = table_width;
    p.table_keys = std::min<int64_t>(table_width * cache->page_size, INT32_MAX);  // (places are 32-bit)
    p.n_pages = cache->n_pages;
    p.page_stride = cache->page_stride;
    p.token_stride = cache->token_stride;
    p.head_stride = cache->head_stride;
    p.B = B;
    p.page_size = cache->page_size;
    p.page_shift = log2_or_none(cache->page_size);
    p.status = device_status_ptr();
    ProfScope ps("ra_kv_cache_append", static_cast<cudaStream_t>(stream));
    const cudaError_t e = launch_rope(p, dt, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? RA_OK : launch_failed(e, "cache append launch");
}

size_t ra_paged_attn_workspace_bytes(int64_t T, int B, int n_groups, int Hq, int Hkv, int d, int dtype,
                                     int max_q_len) {
    if (check_paged_shape(T, B, n_groups, Hq, Hkv, d, dtype)) return 0;
    return paged_layout(T, B, n_groups, Hq / Hkv, Hkv, d, dtype, max_q_len).bytes;
}

ra_status ra_paged_attn_fwd(const void *q, int64_t q_stride, int64_t T, int Hq, const ra_paged_kv *cache,
                            const int32_t *page_table, int64_t table_width, const int32_t *cu_seqlens_q,
                            const int32_t *kv_lens, int B, const int32_t *prefix_table, int64_t prefix_width,
                            const int32_t *prefix_lens, const int32_t *prefix_groups, int n_groups, int causal,
                            int max_q_len, float scale, void *out, int out_dtype, float *lse, void *workspace,
                            size_t ws_bytes, void *stream) {
    ra_status st = check_cache(cache);
    if (st) return st;
    const int Hkv = cache->Hkv, d = cache->d, dtype = cache->dtype;
    if ((st = check_paged_shape(T, B, n_groups, Hq, Hkv, d, dtype))) return st;
    if (out_dtype != RA_FP32 && out_dtype != dtype)
        return fail(RA_ERR_INVALID_ARG, "out_dtype must be RA_FP32 or the cache's dtype");
    const float scale_log2 = scale * 1.4426950408889634f;
    if (!std::isfinite(scale_log2)) return fail(RA_ERR_INVALID_ARG, "scale must be finite, also times log2(e)");
    if (table_width < 0 || prefix_width < 0 || table_width > INT32_MAX || prefix_width > INT32_MAX)
        return fail(RA_ERR_INVALID_ARG, "table widths must be in [0, 2^31)");
    if (q_stride < (int64_t)Hq * d) return fail(RA_ERR_INVALID_ARG, "q_stride is smaller than the heads");
    if (T == 0) return RA_OK;
    if (!q || !out || !lse || !cu_seqlens_q || !kv_lens || (table_width > 0 && !page_table) ||
        (cache->n_pages > 0 && (!cache->k || !cache->v)))
        return fail(RA_ERR_INVALID_ARG, "NULL pointer");
    if (n_groups > 0 && (!prefix_lens || !prefix_groups || (prefix_width > 0 && !prefix_table)))
        return fail(RA_ERR_INVALID_ARG, "a prefix array is NULL");
    const int64_t vec = 16 / elem(dtype);
    if (!on16(q) || !on16(out) || !on16(cache->k) || !on16(cache->v) || q_stride % vec || cache->page_stride % vec ||
        cache->token_stride % vec || cache->head_stride % vec)
        return fail(RA_ERR_UNSUPPORTED, "q, out and the cache must be 16-byte aligned, with strides of whole 16 bytes");
    const PagedLayout L = paged_layout(T, B, n_groups, Hq / Hkv, Hkv, d, dtype, max_q_len);
    if (!workspace || ws_bytes < L.bytes)
        return fail(RA_ERR_WORKSPACE, "workspace must be >= " + std::to_string(L.bytes));
    if (reinterpret_cast<uintptr_t>(workspace) & 255u)
        return fail(RA_ERR_UNSUPPORTED, "workspace must be 256-byte aligned");
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    PagedArgs a{};
    a.q = q;
    a.q_stride = q_stride;
    a.T = T;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.G = Hq / Hkv;
    a.d = d;
    a.dtype = dtype;
    a.k = cache->k;
    a.v = cache->v;
    a.n_pages = cache->n_pages;
    a.page_stride = cache->page_stride;
    a.token_stride = cache->token_stride;
    a.head_stride = cache->head_stride;
    a.page_size = cache->page_size;
    a.page_shift = log2_or_none(cache->page_size);
    if (a.G > 1) a.G_inv = ~0ull / (unsigned)a.G + 1;
    a.B = B;
    a.n_groups = n_groups;
    a.causal = causal != 0;
    a.cu = cu_seqlens_q;
    a.kv_lens = kv_lens;
    a.prefix_lens = prefix_lens;
    a.groups = prefix_groups;
    a.scale_log2 = scale_log2;
    enum { kSimt, kMma, kWide } kind[2];
    int64_t most[2];   // query rows of a segment per KV head
    double passes[2];  // of 64 rows over tiles of 64 keys, at most: what the warp-level kernel would make
    bool want = false;
    for (int f = 0; f < 2; ++f) {
        PagedFamily &F = a.f[f];
        F.S = f ? n_groups : B;
        // (a cache without pages holds no keys: every length above 0 is out of range)
        F.width = cache->n_pages == 0 ? 0 : f ? prefix_width : table_width;
        most[f] = paged_rows(f, T, a.G, max_q_len);
        const int64_t tiles = (most[f] + 63) / 64;  // (a family's prefixes share its rows)
        passes[f] = (double)Hkv * (f ? std::max<int64_t>(F.S, tiles) : F.S * tiles) * ((F.width * cache->page_size + 63) / 64);
        // The kernel: what one warp-level pass over the keys holds, else the tcgen05 kernel's where there is enough to
        // do (it starts 4 us later).  Measured, own keys of 24 sequences, 24 rows: warp-level 44 us, tcgen05 50; 48
        // rows: 61 and 59; 64 rows: 74 and 70, 64 sequences of one KV head 27.6 and 22.4.  A prefix for 8 KV heads, 32
        // rows: 8000 keys 22.8 and 23.6, 30000 keys 36.5 and 35.5; 64 rows: 2000 keys 22.5 and 23.9, 4000 26.6 and
        // 26.0, 8000 34.3 and 30.2; 256 rows: 1000 keys 24.5 and 25.5, 2000 30.7 and 28.2.
        kind[f] = !paged_mma_supported(dtype, d) ? kSimt
                  : F.S && most[f] > (f ? 16 : 32) && passes[f] > (most[f] <= 32 ? 12 : 3) * (double)paged_sms() ? kWide
                                                                                                                  : kMma;
        want = want || kind[f] == kWide;
    }
    PagedMaps maps;
    const bool wide = want && paged_tc_maps(a, maps);
    for (int f = 0; f < 2; ++f) {
        PagedFamily &F = a.f[f];
        if (kind[f] == kWide && !wide) kind[f] = kMma;
        F.rt = kind[f] == kWide ? kPagedWideRows : most[f] <= 16 ? 16 : kind[f] == kMma && most[f] <= 32 ? 32 : 64;
        // The SIMT kernel with few 64-row tiles: four times as many of a quarter, while an SM has one of them at d > 64
        // and four below.  fp32, 64 and 16 rows a tile: 1000 keys of 2 heads of 128, 32 rows, 17.5 and 15.0 us; 4
        // sequences of 500, 64 rows, 21.8 and 28; 4000 keys of 64, 64 rows, 19.4 and 16.4.
        if (kind[f] == kSimt && 4 * passes[f] <= paged_sms() * (d <= 64 ? 4 : 1)) F.rt = 16;
        F.kt = kind[f] == kWide ? 128 : 64;
        while (1 << F.rt_log < F.rt) ++F.rt_log;
        while (1 << F.kt_log < F.kt) ++F.kt_log;
        F.halves = kind[f] == kWide;
        // The shortest run, in sixteenths of a warp-level tile: two tiles where a partial has 32 rows or more, whose
        // write and join cost about a tile.  8192 keys of one KV head, 32 rows with 1 and 2 tiles at least: 14.8 and
        // 12.4 us; the tcgen05 kernel, 128 rows: 17.3 with 1, 15.9 with 2, 15.6 with 4 (1024 keys: 9.8, 10.6, 12.7).
        // With 16 rows one or two makes no difference.
        F.least = kind[f] == kWide ? 64 : kind[f] == kMma && F.rt > 16 ? 32 : 16;
        if (F.S)
            F.n = kind[f] == kWide  ? std::min(kPagedMaxWide, paged_sms())
                  : kind[f] == kMma ? paged_mma_ctas(F.rt, d, cache->page_size)
                                    : paged_simt_ctas(F.rt, d);
        F.seg = reinterpret_cast<PagedSeg *>(ws + L.o_seg[f]);
        F.hdr = reinterpret_cast<PagedHdr *>(ws + L.o_hdr[f]);
        F.start = reinterpret_cast<int *>(ws + L.o_start[f]);
        F.table = f ? prefix_table : page_table;
        F.acc = reinterpret_cast<float *>(ws + L.o_acc[f]);
        F.ml = reinterpret_cast<float *>(ws + L.o_ml[f]);
    }
    a.out = out;
    a.out_dtype = out_dtype;
    a.lse = lse;
    a.status = device_status_ptr();
    cudaError_t e;
    a.here = B <= kPagedHere && n_groups <= kPagedHere;
    if (!a.here) {
        ProfScope ps("ra_paged_plan", s);
        if ((e = launch_paged_plan(a, s)) != cudaSuccess) return launch_failed(e, "paged plan launch");
    }
    for (int f = 1; f >= 0; --f) {
        if (a.f[f].S == 0) continue;
        ProfScope ps(f ? "ra_paged_prefix" : "ra_paged_own", s);
        const int late = f == 0 && n_groups > 0;  // behind the prefixes' kernel, and independent of it
        e = kind[f] == kWide  ? launch_paged_tc(a, f, late, maps, s)
            : kind[f] == kMma ? launch_paged_mma(a, f, late, s)
                              : launch_paged_simt(a, f, late, s);
        if (e != cudaSuccess) return launch_failed(e, "paged attention launch");
    }
    ProfScope ps("ra_paged_combine", s);
    if ((e = launch_paged_combine(a, s)) != cudaSuccess) return launch_failed(e, "paged combine launch");
    return RA_OK;
}

}  // extern "C"

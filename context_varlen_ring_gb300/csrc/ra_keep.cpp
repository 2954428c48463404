// ra_keep.cpp -- the C entries of what keeps the paged cache within a budget:
// the weights that its keys gather, and eviction by them.  Argument checks and
// the choice of kernels; host code only.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <string>

#include "ra_internal.h"
#include "ra_keep.h"
#include "ra_kernels.h"

namespace ra {
namespace {

bool on16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int log2_or_none(int x) {
    for (int i = 0; i < 31; ++i)
        if (x == 1 << i) return i;
    return -1;
}

// Whether places that are written have memory of their own (strides of 0, as an expanded tensor has them, share it).
bool apart(const ra_paged_kv *c, int64_t page, int64_t token, int64_t head) {
    return (page != 0 || c->n_pages <= 1) && (token != 0 || c->page_size <= 1) && (head != 0 || c->Hkv <= 1);
}

// The cache's shape, and weights on the same pages.
ra_status check_pages(const ra_paged_kv *c, const ra_paged_weights *w) {
    if (!c || !w) return fail(RA_ERR_INVALID_ARG, "cache or weights is NULL");
    if (c->dtype != RA_BF16 && c->dtype != RA_FP32)
        return fail(RA_ERR_INVALID_ARG, "the cache's dtype must be RA_BF16 or RA_FP32");
    if (c->n_pages < 0 || c->n_pages > INT32_MAX || c->page_size < 1 || c->Hkv < 1 || c->Hkv > 4096 || c->d < 1)
        return fail(RA_ERR_INVALID_ARG, "bad cache shape");
    if (c->page_stride < 0 || c->token_stride < 0 || c->head_stride < 0 || w->page_stride < 0 || w->token_stride < 0 ||
        w->head_stride < 0)
        return fail(RA_ERR_INVALID_ARG, "the strides must not be negative");
    const int vec = c->dtype == RA_FP32 ? 4 : 8;
    if (c->d % vec || c->d > 256) return fail(RA_ERR_UNSUPPORTED, "d must be whole 16 bytes and <= 256");
    if (!on16(c->k) || !on16(c->v) || c->page_stride % vec || c->token_stride % vec || c->head_stride % vec)
        return fail(RA_ERR_UNSUPPORTED, "the cache must be 16-byte aligned, with strides of whole 16 bytes");
    if (reinterpret_cast<uintptr_t>(w->w) & 3u) return fail(RA_ERR_UNSUPPORTED, "the weights are not aligned");
    if (c->n_pages > 0 && !w->w) return fail(RA_ERR_INVALID_ARG, "the weights are NULL");
    if (!apart(c, w->page_stride, w->token_stride, w->head_stride))
        return fail(RA_ERR_INVALID_ARG, "weights must not share memory (a stride of 0)");
    return RA_OK;
}

}  // namespace
}  // namespace ra

using namespace ra;

extern "C" {

ra_status ra_paged_attn_key_weights(const void *q, int64_t q_stride, int64_t T, int Hq, const ra_paged_kv *cache,
                                    const ra_paged_weights *weights, const int32_t *page_table, int64_t table_width,
                                    const int32_t *cu_seqlens_q, const int32_t *kv_lens, int B,
                                    const int32_t *prefix_table, int64_t prefix_width, const int32_t *prefix_lens,
                                    const int32_t *prefix_groups, int n_groups, int causal, int max_q_len, float scale,
                                    const float *lse, void *stream) {
    ra_status st = check_pages(cache, weights);
    if (st) return st;
    const int Hkv = cache->Hkv, d = cache->d;
    if (T < 0 || n_groups < 0 || B < 0 || (B == 0 && T > 0))
        return fail(RA_ERR_INVALID_ARG, "T and n_groups must be >= 0, B >= 1 (0 with T = 0: an empty batch)");
    if (Hq <= 0 || Hq % Hkv != 0) return fail(RA_ERR_INVALID_ARG, "Hq must be a positive multiple of Hkv");
    if (d % 32 != 0) return fail(RA_ERR_UNSUPPORTED, "d must be a multiple of 32 and <= 256");
    if (T > (1 << 30) / Hq) return fail(RA_ERR_UNSUPPORTED, "T * Hq must be at most 2^30");
    if (B > (1 << 20) || n_groups > (1 << 20)) return fail(RA_ERR_UNSUPPORTED, "too many sequences");
    const float scale_log2 = scale * 1.4426950408889634f;
    if (!std::isfinite(scale_log2)) return fail(RA_ERR_INVALID_ARG, "scale must be finite, also times log2(e)");
    if (table_width < 0 || prefix_width < 0 || table_width > INT32_MAX || prefix_width > INT32_MAX)
        return fail(RA_ERR_INVALID_ARG, "table widths must be in [0, 2^31)");
    if (q_stride < (int64_t)Hq * d) return fail(RA_ERR_INVALID_ARG, "q_stride is smaller than the heads");
    if (T == 0) return RA_OK;
    if (!q || !lse || !cu_seqlens_q || !kv_lens || (table_width > 0 && !page_table) || (cache->n_pages > 0 && !cache->k))
        return fail(RA_ERR_INVALID_ARG, "NULL pointer");
    if (n_groups > 0 && (!prefix_lens || !prefix_groups || (prefix_width > 0 && !prefix_table)))
        return fail(RA_ERR_INVALID_ARG, "a prefix array is NULL");
    if (!on16(q) || q_stride % (cache->dtype == RA_FP32 ? 4 : 8))
        return fail(RA_ERR_UNSUPPORTED, "q must be 16-byte aligned, with a stride of whole 16 bytes");
    WeightArgs a{};
    a.q = q;
    a.q_stride = q_stride;
    a.T = T;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.G = Hq / Hkv;
    a.d = d;
    a.dtype = cache->dtype;
    a.k = cache->k;
    a.n_pages = cache->n_pages;
    a.page_stride = cache->page_stride;
    a.token_stride = cache->token_stride;
    a.head_stride = cache->head_stride;
    a.w = weights->w;
    a.w_page = weights->page_stride;
    a.w_token = weights->token_stride;
    a.w_head = weights->head_stride;
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
    a.table[0] = page_table;
    a.table[1] = prefix_table;
    a.width[0] = cache->n_pages == 0 ? 0 : table_width;  // (a cache without pages holds no keys)
    a.width[1] = cache->n_pages == 0 ? 0 : prefix_width;
    a.scale_log2 = scale_log2;
    a.lse = lse;
    a.status = device_status_ptr();
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    ProfScope ps("ra_paged_attn_key_weights", s);
    cudaError_t e;
    if (weights_mma_supported(a.dtype, d)) {
        // The kernel, by the query rows that a KV head may have and the keys that the tables have room for.  Few rows:
        // the stream (up to 32 rows of 8 sequences of 2000 keys the tiles are faster, 22.6 us to its 28.3).  From 64 rows
        // on tcgen05, where there are a few tiles of 256 keys (15 sequences of 5 tokens behind a prefix 12.3 us, by tiles of
        // 64 keys 26.7; 4 of 200 tokens and 1000 keys of 2 heads 18.6 and 38.9; with prefixes one kernel takes own keys and
        // shared ones: 64 single tokens, up to 8192 own keys behind 32768, 118 us, by tiles of 64 keys 209, by the stream
        // 1187).  Else tiles of 64 keys, or of fewer where
        // those would leave SMs without one: 500 keys of 8 heads by tiles of 64, 32 and 16 keys 12.3, 10.3 and 8.2 us, 3000
        // of 2 heads (groups of 7) 82, 68 and 52; 2000 of 8 in 8 sequences 22.6, 26.7 and 45.
        const int64_t rows = (max_q_len > 0 && n_groups == 0 ? std::min<int64_t>(max_q_len, T) : T) * a.G;
        auto tiles = [&](int keys) {
            return Hkv * (B * ((a.width[0] * a.page_size + keys - 1) / keys) + n_groups * ((a.width[1] * a.page_size + keys - 1) / keys));
        };
        PagedMaps maps;
        if (rows <= 16)
            e = launch_weights_stream(a, s);
        else if (rows >= 64 && tiles(256) >= 8 && weights_tc_maps(a, maps))
            e = launch_weights_tc(a, maps, s);
        else
            e = launch_weights_mma(a, tiles(64) < paged_sms() ? 16 : tiles(64) < 2 * paged_sms() ? 32 : 64, s);
    } else {
        e = launch_weights_simt(a, s);
    }
    return e == cudaSuccess ? RA_OK : fail(RA_ERR_CUDA, std::string("key weights launch: ") + cudaGetErrorString(e));
}

ra_status ra_kv_cache_evict(const ra_paged_kv *cache, const ra_paged_weights *weights, const int32_t *page_table,
                            int64_t table_width, const int32_t *kv_lens, int B, int keep, const int32_t *keep_lens,
                            int sinks, int recent, int per_head, const int32_t *out_table, int64_t out_width,
                            int32_t *new_lens, int32_t *kept, void *stream) {
    ra_status st = check_pages(cache, weights);
    if (st) return st;
    if (!apart(cache, cache->page_stride, cache->token_stride, cache->head_stride))
        return fail(RA_ERR_INVALID_ARG, "the cache's rows must not share memory (a stride of 0)");
    if (B < 0 || B > (1 << 20) || (int64_t)B * cache->Hkv > (1 << 26))
        return fail(RA_ERR_INVALID_ARG, "B must be in [0, 2^20] and B * Hkv at most 2^26");
    if (keep < 1 || keep > (1 << 30)) return fail(RA_ERR_INVALID_ARG, "keep must be in [1, 2^30]");
    if (sinks < 0 || recent < 0 || (int64_t)sinks + recent > keep)
        return fail(RA_ERR_INVALID_ARG, "sinks and recent must be >= 0 and at most keep together");
    if (table_width < 0 || table_width > INT32_MAX || out_width < 0 || out_width > INT32_MAX)
        return fail(RA_ERR_INVALID_ARG, "table widths must be in [0, 2^31)");
    if (B == 0) return RA_OK;
    if (!kv_lens || !new_lens || !kept || (table_width > 0 && !page_table) || (cache->n_pages > 0 && (!cache->k || !cache->v)))
        return fail(RA_ERR_INVALID_ARG, "NULL pointer");
    if (new_lens == kv_lens) return fail(RA_ERR_INVALID_ARG, "new_lens must not be kv_lens");
    EvictArgs a{};
    a.k = cache->k;
    a.v = cache->v;
    a.n_pages = cache->n_pages;
    a.page_stride = cache->page_stride;
    a.token_stride = cache->token_stride;
    a.head_stride = cache->head_stride;
    a.w = weights->w;
    a.w_page = weights->page_stride;
    a.w_token = weights->token_stride;
    a.w_head = weights->head_stride;
    a.page_size = cache->page_size;
    a.page_shift = log2_or_none(cache->page_size);
    a.Hkv = cache->Hkv;
    a.esize = cache->dtype == RA_FP32 ? 4 : 2;
    a.row_bytes = cache->d * a.esize;
    a.table = page_table;
    a.width = table_width;
    a.most = cache->n_pages == 0 ? 0 : std::min<int64_t>(table_width * cache->page_size, 1 << 30);
    a.kv_lens = kv_lens;
    a.B = B;
    a.H = per_head ? cache->Hkv : 1;
    a.keep = keep;
    a.sinks = sinks;
    a.recent = recent;
    a.keep_lens = keep_lens;
    a.out_table = out_table;
    a.out_width = out_width;
    a.new_lens = new_lens;
    a.kept = kept;
    a.status = device_status_ptr();
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    {
        ProfScope ps("ra_evict_choose", s);
        if ((e = launch_evict_choose(a, s)) != cudaSuccess)
            return fail(RA_ERR_CUDA, std::string("eviction's choice launch: ") + cudaGetErrorString(e));
    }
    ProfScope ps("ra_evict_move", s);
    if ((e = launch_evict_move(a, s)) != cudaSuccess)
        return fail(RA_ERR_CUDA, std::string("eviction's move launch: ") + cudaGetErrorString(e));
    return RA_OK;
}

}  // extern "C"

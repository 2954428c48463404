// ra_keep.h -- arguments of the kernels that keep the paged cache within a
// budget: the attention weight that its keys gather (ra_weights.cu) and
// eviction by it (ra_evict.cu); filled by the C entries in ra_keep.cpp.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace ra {

struct WeightArgs {
    const void *q;
    int64_t q_stride, T;
    int Hq, Hkv, G, d, dtype;
    const void *k;
    int64_t n_pages, page_stride, token_stride, head_stride;
    float *w;                          // the same pages and rows, [.., heads]
    int64_t w_page, w_token, w_head;
    int page_size, page_shift;         // page_shift: its log2, or -1
    unsigned long long G_inv;          // 2^64 / G, rounded up (G > 1)
    int B, n_groups, causal;
    const int32_t *cu, *kv_lens, *prefix_lens, *groups;
    const int32_t *table[2];           // of the sequences, of the prefixes
    int64_t width[2];
    float scale_log2;
    const float *lse;                  // [Hq, T]
    int *status;
};
bool weights_mma_supported(int dtype, int d);
cudaError_t launch_weights_mma(const WeightArgs &a, int keys, cudaStream_t st);   // keys a unit: 16, 32 or 64
cudaError_t launch_weights_stream(const WeightArgs &a, cudaStream_t st);  // few query rows (as weights_mma_supported)
cudaError_t launch_weights_simt(const WeightArgs &a, cudaStream_t st);

struct PagedMaps;
bool weights_tc_maps(const WeightArgs &a, PagedMaps &m);  // false: not a shape of the tcgen05 kernel
cudaError_t launch_weights_tc(const WeightArgs &a, const PagedMaps &m, cudaStream_t st);

struct EvictArgs {
    void *k, *v;
    int64_t n_pages, page_stride, token_stride, head_stride;
    float *w;
    int64_t w_page, w_token, w_head;
    int page_size, page_shift, Hkv, row_bytes, esize;
    const int32_t *table, *kv_lens;
    int64_t width, most;               // entries of a table's row; the keys that they hold (lengths are 32-bit)
    int B, H, keep, sinks, recent;     // H: choices a sequence (Hkv, or 1 for all heads)
    const int32_t *keep_lens;          // [B] or NULL
    const int32_t *out_table;          // NULL: in place
    int64_t out_width;
    int32_t *new_lens, *kept;          // [B], [B, H, keep]
    int *status;
};
cudaError_t launch_evict_choose(const EvictArgs &a, cudaStream_t st);
cudaError_t launch_evict_move(const EvictArgs &a, cudaStream_t st);

}  // namespace ra

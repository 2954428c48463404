// ra_delta.h -- arguments of the gated delta rule's kernels (ra_delta.cu,
// ra_delta_bwd.cu), filled by the C entries in ra_delta.cpp.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace ra {

constexpr int kDeltaChunk = 64;        // tokens a chunk
constexpr int kDeltaParts = 3;         // bf16 parts of what is not bf16 itself

// A chunk: its first token, its tokens (1 .. 64).
struct DeltaChunk {
    int tok0, n;
};
struct DeltaHdr {
    int chunks, bad, pad[2];
};
struct DeltaArgs {
    const void *q, *k, *v;             // rows of Hk * dk, Hk * dk, Hv * dv elements
    int64_t q_stride, k_stride, v_stride;
    const float *g, *beta;             // [T, Hv]
    int dtype, Hk, Hv, dk, dv, N;
    int64_t T;
    const int32_t *cu;                 // DEVICE [N + 1]
    float scale;
    const float *state;                // [n_slots, Hv, dk, dv] or NULL (zeros)
    float *state_out;                  // [n_slots, Hv, dk, dv] or NULL
    const int32_t *slots;              // [N] or NULL (the sequence's number)
    int64_t n_slots;
    void *out;                         // [T, Hv, dv]; NULL: not wanted
    int max_chunks;                    // no boundaries of T tokens in N sequences give more
    // workspace
    DeltaHdr *hdr;
    DeltaChunk *chunk;                 // [max_chunks]
    int *first, *order;                // [N + 1] the sequences' first chunks, [N] sequences, most chunks first
    uint16_t *tp;                      // [max_chunks][Hv][2][parts][64][64] bf16: T and P
    float *s0, *ds;                    // [max_chunks][Hv][dk][dv]: state ahead of each chunk, gradient of that behind it
    float *u, *r, *dr;                 // [max_chunks][Hv][64][dv]
    // backward
    const void *dout;
    int64_t dout_stride;
    const float *dstate;               // [N, Hv, dk, dv] or NULL (zeros)
    float *dstate0;                    // [N, Hv, dk, dv] or NULL
    void *dq, *dk_, *dv_;              // [T, Hk, dk], [T, Hk, dk], [T, Hv, dv]
    float *dg, *dbeta;                 // [T, Hv]
    float *part;                       // [2][T][Hv][dk] fp32 gradients of each value head; NULL where the kernel that
                                       // makes them has their sums (Hv == Hk, or delta_tc_shape)
    int *status;
};

// The types and heads of the kernels on tcgen05, which sum a key head's gradients by themselves.
constexpr bool delta_tc_shape(bool bf16, int dk, int dv) { return bf16 && dk == 128 && dv == 128; }

cudaError_t launch_delta_plan(const DeltaArgs &a, cudaStream_t st);
cudaError_t launch_delta_local(const DeltaArgs &a, cudaStream_t st);   // T and P of every chunk
cudaError_t launch_delta_scan(const DeltaArgs &a, int keep, cudaStream_t st);  // keep: s0, u and r for the backward
bool delta_tc_supported(const DeltaArgs &a);  // the walks on tcgen05 (ra_delta_tc.cu)
cudaError_t launch_delta_tc_scan(const DeltaArgs &a, cudaStream_t st);   // launch_delta_scan that keeps nothing
cudaError_t launch_delta_tc_walks(const DeltaArgs &a, cudaStream_t st);  // launch_delta_scan that keeps, and launch_delta_back
cudaError_t launch_delta_tc_grads(const DeltaArgs &a, cudaStream_t st);  // launch_delta_grads
cudaError_t launch_delta_back(const DeltaArgs &a, cudaStream_t st);    // ds, dr and dv, chunk by chunk from the end
cudaError_t launch_delta_grads(const DeltaArgs &a, cudaStream_t st);   // dq, dk, dg, dbeta of every chunk
cudaError_t launch_delta_sum(const DeltaArgs &a, cudaStream_t st);     // dq and dk over a key head's value heads

struct DeltaStepArgs {
    const void *q, *k, *v;             // [B, Hk, dk], [B, Hk, dk], [B, Hv, dv]
    int64_t q_stride, k_stride, v_stride;
    const float *g, *beta;             // [B, Hv]
    int dtype, Hk, Hv, dk, dv, B;
    float scale;
    float *state;                      // [n_slots, Hv, dk, dv]
    const int32_t *slots;
    int64_t n_slots;
    void *out;
    int *status;
};
cudaError_t launch_delta_step(const DeltaStepArgs &a, cudaStream_t st);

}  // namespace ra

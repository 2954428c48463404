// ra_delta.cpp -- the C entries of the gated delta rule: argument checks,
// workspace layout and the order of the kernels.  Host code only.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <string>

#include "ra_delta.h"
#include "ra_internal.h"
#include "ra_kernels.h"

namespace ra {
namespace {

bool on16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// What the sizes alone decide.
ra_status check_shape(int64_t T, int64_t N, int Hk, int Hv, int dk, int dv, int dtype) {
    if (dtype != RA_BF16 && dtype != RA_FP32) return fail(RA_ERR_INVALID_ARG, "dtype must be RA_BF16 or RA_FP32");
    if (T < 0 || N < 0 || (N == 0 && T > 0))
        return fail(RA_ERR_INVALID_ARG, "T must be >= 0 and N >= 1 (0 with T = 0: an empty batch)");
    if (Hk <= 0 || Hv <= 0 || Hv % Hk != 0) return fail(RA_ERR_INVALID_ARG, "Hv must be a positive multiple of Hk");
    if ((dk != 64 && dk != 128) || (dv != 64 && dv != 128))
        return fail(RA_ERR_UNSUPPORTED, "dk and dv must be 64 or 128");
    if (Hv > 4096 || T > (1 << 30) || N > (1 << 20) || N * Hv > (1 << 26))
        return fail(RA_ERR_UNSUPPORTED, "too many heads, tokens or sequences");
    return RA_OK;
}

ra_status check_inputs(const ra_delta *d) {
    const int e = d->dtype == RA_FP32 ? 4 : 2;
    if (d->T > 0 && (!d->q || !d->k || !d->v || !d->g || !d->beta)) return fail(RA_ERR_INVALID_ARG, "NULL pointer");
    if (d->T > 0 && (d->q_stride < (int64_t)d->Hk * d->dk || d->k_stride < (int64_t)d->Hk * d->dk ||
                     d->v_stride < (int64_t)d->Hv * d->dv))
        return fail(RA_ERR_INVALID_ARG, "a row stride is smaller than its heads");
    if (!on16(d->q) || !on16(d->k) || !on16(d->v) || !on16(d->state) ||
        (d->T > 1 && (d->q_stride * e % 16 || d->k_stride * e % 16 || d->v_stride * e % 16)))
        return fail(RA_ERR_UNSUPPORTED, "q, k, v and the states must be 16-byte aligned, with strides of whole 16 bytes");
    if (!std::isfinite(d->scale)) return fail(RA_ERR_INVALID_ARG, "scale must be finite");
    return RA_OK;
}

int64_t most_chunks(int64_t T, int64_t N) { return T / kDeltaChunk + std::min(T, N); }

struct Layout {
    size_t hdr, chunk, first, order, tp, s0, ds, u, r, dr, part, bytes;
};
Layout layout(int64_t T, int64_t N, int Hk, int Hv, int dk, int dv, int dtype, int bwd) {
    Layout L{};
    size_t at = 0;
    auto take = [&](size_t n) {
        const size_t o = at;
        at = align_up(at + n, 256);
        return o;
    };
    const size_t cells = (size_t)most_chunks(T, N) * Hv;
    L.hdr = take(sizeof(DeltaHdr));
    L.chunk = take((size_t)most_chunks(T, N) * sizeof(DeltaChunk));
    L.first = take((size_t)(N + 1) * 4);
    L.order = take((size_t)N * 4);
    L.tp = take(cells * 2 * kDeltaParts * kDeltaChunk * kDeltaChunk * 2);
    if (bwd) {
        L.s0 = take(cells * dk * dv * 4);
        L.ds = take(cells * dk * dv * 4);
        L.u = take(cells * kDeltaChunk * dv * 4);
        L.r = take(cells * kDeltaChunk * dv * 4);
        L.dr = take(cells * kDeltaChunk * dv * 4);
        if (Hv != Hk && !delta_tc_shape(dtype == RA_BF16, dk, dv)) L.part = take((size_t)T * Hv * dk * 4 * 2);
    }
    L.bytes = at;
    return L;
}

DeltaArgs arguments(const ra_delta *d, uint8_t *ws, const Layout &L, int bwd) {
    DeltaArgs a{};
    a.q = d->q;
    a.k = d->k;
    a.v = d->v;
    a.q_stride = d->q_stride;
    a.k_stride = d->k_stride;
    a.v_stride = d->v_stride;
    a.g = d->g;
    a.beta = d->beta;
    a.dtype = d->dtype;
    a.Hk = d->Hk;
    a.Hv = d->Hv;
    a.dk = d->dk;
    a.dv = d->dv;
    a.N = d->N;
    a.T = d->T;
    a.cu = d->cu_seqlens;
    a.scale = d->scale;
    a.state = d->state;
    a.slots = d->slots;
    a.n_slots = d->n_slots;
    a.max_chunks = (int)most_chunks(d->T, d->N);
    a.hdr = reinterpret_cast<DeltaHdr *>(ws + L.hdr);
    a.chunk = reinterpret_cast<DeltaChunk *>(ws + L.chunk);
    a.first = reinterpret_cast<int *>(ws + L.first);
    a.order = reinterpret_cast<int *>(ws + L.order);
    a.tp = reinterpret_cast<uint16_t *>(ws + L.tp);
    if (bwd) {
        a.s0 = reinterpret_cast<float *>(ws + L.s0);
        a.ds = reinterpret_cast<float *>(ws + L.ds);
        a.u = reinterpret_cast<float *>(ws + L.u);
        a.r = reinterpret_cast<float *>(ws + L.r);
        a.dr = reinterpret_cast<float *>(ws + L.dr);
        if (L.part) a.part = reinterpret_cast<float *>(ws + L.part);
    }
    a.status = device_status_ptr();
    return a;
}

ra_status check_call(const ra_delta *d, const Layout &L, const void *workspace, size_t ws_bytes) {
    if (!d->cu_seqlens) return fail(RA_ERR_INVALID_ARG, "cu_seqlens is NULL");
    if (d->state && d->n_slots < 0) return fail(RA_ERR_INVALID_ARG, "n_slots must be >= 0");
    if (d->state && !d->slots && d->n_slots < d->N)
        return fail(RA_ERR_INVALID_ARG, "without slots there must be a state for each sequence");
    if (!workspace || ws_bytes < L.bytes)
        return fail(RA_ERR_WORKSPACE, "workspace must be >= " + std::to_string(L.bytes));
    if (reinterpret_cast<uintptr_t>(workspace) & 255u)
        return fail(RA_ERR_UNSUPPORTED, "workspace must be 256-byte aligned");
    return RA_OK;
}

ra_status launched(cudaError_t e, const char *what) {
    return e == cudaSuccess ? RA_OK : fail(RA_ERR_CUDA, std::string(what) + " launch: " + cudaGetErrorString(e));
}

template <typename F>
ra_status step(const char *name, cudaStream_t s, F &&f) {
    ProfScope ps(name, s);
    return launched(f(), name);
}

}  // namespace
}  // namespace ra

using namespace ra;

extern "C" {

size_t ra_delta_rule_workspace_bytes(int64_t T, int N, int Hk, int Hv, int dk, int dv, int dtype, int bwd) {
    if (check_shape(T, N, Hk, Hv, dk, dv, dtype)) return 0;
    return layout(T, N, Hk, Hv, dk, dv, dtype, bwd).bytes;
}

ra_status ra_delta_rule_fwd(const ra_delta *d, void *out, float *state_out, void *workspace, size_t ws_bytes,
                            void *stream) {
    if (!d) return fail(RA_ERR_INVALID_ARG, "d is NULL");
    ra_status st = check_shape(d->T, d->N, d->Hk, d->Hv, d->dk, d->dv, d->dtype);
    if (st || (st = check_inputs(d))) return st;
    if (d->N == 0 || (d->T == 0 && !state_out)) return RA_OK;
    if (d->T > 0 && !out) return fail(RA_ERR_INVALID_ARG, "out is NULL");
    if (!on16(out) || !on16(state_out)) return fail(RA_ERR_UNSUPPORTED, "out and state_out must be 16-byte aligned");
    if (state_out && (d->n_slots < 0 || (!d->slots && d->n_slots < d->N)))
        return fail(RA_ERR_INVALID_ARG, "without slots there must be a state for each sequence");
    const Layout L = layout(d->T, d->N, d->Hk, d->Hv, d->dk, d->dv, d->dtype, 0);
    if ((st = check_call(d, L, workspace, ws_bytes))) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    DeltaArgs a = arguments(d, static_cast<uint8_t *>(workspace), L, 0);
    a.out = out;
    a.state_out = state_out;
    if ((st = step("ra_delta_plan", s, [&] { return launch_delta_plan(a, s); }))) return st;
    if (a.max_chunks > 0 && (st = step("ra_delta_local", s, [&] { return launch_delta_local(a, s); }))) return st;
    return step("ra_delta_scan", s, [&] { return delta_tc_supported(a) ? launch_delta_tc_scan(a, s) : launch_delta_scan(a, 0, s); });
}

ra_status ra_delta_rule_bwd(const ra_delta *d, const void *dout, int64_t dout_stride, const float *dstate, void *dq,
                            void *dk, void *dv, float *dg, float *dbeta, float *dstate0, void *workspace,
                            size_t ws_bytes, void *stream) {
    if (!d) return fail(RA_ERR_INVALID_ARG, "d is NULL");
    ra_status st = check_shape(d->T, d->N, d->Hk, d->Hv, d->dk, d->dv, d->dtype);
    if (st || (st = check_inputs(d))) return st;
    if (d->N == 0 || (d->T == 0 && !dstate0)) return RA_OK;
    if (d->T > 0 && (!dout || !dq || !dk || !dv || !dg || !dbeta)) return fail(RA_ERR_INVALID_ARG, "NULL pointer");
    if (d->T > 0 && dout_stride < (int64_t)d->Hv * d->dv)
        return fail(RA_ERR_INVALID_ARG, "the row stride of dout is smaller than its heads");
    const int e = d->dtype == RA_FP32 ? 4 : 2;
    if (!on16(dout) || !on16(dq) || !on16(dk) || !on16(dv) || !on16(dstate) || !on16(dstate0) ||
        (d->T > 1 && dout_stride * e % 16))
        return fail(RA_ERR_UNSUPPORTED, "dout, the gradients and the states must be 16-byte aligned, with strides of whole 16 bytes");
    const Layout L = layout(d->T, d->N, d->Hk, d->Hv, d->dk, d->dv, d->dtype, 1);
    if ((st = check_call(d, L, workspace, ws_bytes))) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    DeltaArgs a = arguments(d, static_cast<uint8_t *>(workspace), L, 1);
    a.dout = dout;
    a.dout_stride = dout_stride;
    a.dstate = dstate;
    a.dstate0 = dstate0;
    a.dq = dq;
    a.dk_ = dk;
    a.dv_ = dv;
    a.dg = dg;
    a.dbeta = dbeta;
    if ((st = step("ra_delta_plan", s, [&] { return launch_delta_plan(a, s); }))) return st;
    if (a.max_chunks > 0 && (st = step("ra_delta_local", s, [&] { return launch_delta_local(a, s); }))) return st;
    if (delta_tc_supported(a)) {
        if ((st = step("ra_delta_walks", s, [&] { return launch_delta_tc_walks(a, s); }))) return st;
    } else {
        if (a.max_chunks > 0 && (st = step("ra_delta_scan", s, [&] { return launch_delta_scan(a, 1, s); }))) return st;
        if ((st = step("ra_delta_back", s, [&] { return launch_delta_back(a, s); })) || a.max_chunks == 0) return st;
    }
    if ((st = step("ra_delta_grads", s, [&] { return delta_tc_supported(a) ? launch_delta_tc_grads(a, s) : launch_delta_grads(a, s); })) || !a.part)
        return st;
    return step("ra_delta_sum", s, [&] { return launch_delta_sum(a, s); });
}

ra_status ra_delta_rule_step(const ra_delta *d, float *state, void *out, void *stream) {
    if (!d) return fail(RA_ERR_INVALID_ARG, "d is NULL");
    ra_status st = check_shape(d->T, d->N, d->Hk, d->Hv, d->dk, d->dv, d->dtype);
    if (st || (st = check_inputs(d))) return st;
    if (d->T != d->N) return fail(RA_ERR_INVALID_ARG, "a step takes one token of each sequence: T must be N");
    if (d->N == 0) return RA_OK;
    if (!state || !out) return fail(RA_ERR_INVALID_ARG, "NULL pointer");
    if (!on16(state) || !on16(out)) return fail(RA_ERR_UNSUPPORTED, "state and out must be 16-byte aligned");
    if (d->n_slots < 0 || (!d->slots && d->n_slots < d->N))
        return fail(RA_ERR_INVALID_ARG, "without slots there must be a state for each sequence");
    DeltaStepArgs a{};
    a.q = d->q;
    a.k = d->k;
    a.v = d->v;
    a.q_stride = d->q_stride;
    a.k_stride = d->k_stride;
    a.v_stride = d->v_stride;
    a.g = d->g;
    a.beta = d->beta;
    a.dtype = d->dtype;
    a.Hk = d->Hk;
    a.Hv = d->Hv;
    a.dk = d->dk;
    a.dv = d->dv;
    a.B = d->N;
    a.scale = d->scale;
    a.state = state;
    a.slots = d->slots;
    a.n_slots = d->n_slots;
    a.out = out;
    a.status = device_status_ptr();
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return ra::step("ra_delta_step", s, [&] { return launch_delta_step(a, s); });
}

}  // extern "C"

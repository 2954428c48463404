// ra_serve.cuh -- what the kernels of rotary positions, the cache append and
// paged attention use beside ra_dev.cuh: the search of a token's segment, bulk
// copies out of shared memory, loads with an L2 policy, and a kernel's launch limits.
#pragma once

#include <cuda_runtime.h>

#include <atomic>

#include "ra_dev.cuh"
#include "ra_paged_split.h"

namespace ra {
namespace dev {

// How many of the n non-decreasing ends are <= t: the segment that holds t.
// The whole warp searches, 32 probes a round (n <= 1024 in two rounds).
__device__ __forceinline__ int segment_of(const int32_t *ends, int n, int64_t t) {
    const int lane = threadIdx.x & 31;
    return search32(n, [&](int lo, int step, int left) {
        const int q = (lane + 1) * step - 1;
        const bool le = q < left && (int64_t)__ldg(ends + lo + q) <= t;
        return __popc(__ballot_sync(0xffffffffu, le));
    });
}

// The L2 policy of data that is read once: it leaves first, so that what stays
// (code, tables, partial results) is not pushed out by it.
__device__ __forceinline__ uint64_t l2_evict_first() {
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
    return p;
}
__device__ __forceinline__ void tma_load_4d_hint(void *dst, const CUtensorMap *m, uint64_t *bar, int c0, int c1, int c2,
                                                 int c3, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%3, %4, %5, %6}], [%2], %7;" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "l"(policy)
        : "memory");
}

// 1-D bulk copy shared -> global (16-byte aligned, whole 16 bytes), in the
// issuing thread's bulk group, and the waits on those groups: until all but the
// last N have read shared memory, or until all are complete.
__device__ __forceinline__ void bulk_store(void *dst, const void *src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_u32(src)), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void bulk_wait_read() {
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

}  // namespace dev

// A kernel's shared-memory opt-in and its CTAs an SM, asked once a device.
class LaunchFit {
  public:
    cudaError_t prepare(const void *kernel, int threads, size_t smem, int *ctas) {
        int dev = -1;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        const bool held = dev >= 0 && dev < 128;
        int n = held ? ctas_[dev].load(std::memory_order_acquire) : 0;
        if (n == 0) {
            e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
            if (e != cudaSuccess) return e;
            e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, smem);
            if (e != cudaSuccess) return e;
            n = n > 0 ? n : 1;
            if (held) ctas_[dev].store(n, std::memory_order_release);
        }
        if (ctas) *ctas = n;
        return cudaSuccess;
    }

  private:
    std::atomic<int> ctas_[128] = {};
};

}  // namespace ra

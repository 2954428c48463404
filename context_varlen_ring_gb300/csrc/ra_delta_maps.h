// ra_delta_maps.h -- the tensor maps of the gated delta rule's tcgen05 kernels.
#pragma once

#include <cuda.h>

#include <cstdint>

namespace ra {

// Rows [T][H][128] of bf16, `stride` elements apart, in boxes of 64 tokens of one head: 64 columns wide with the
// tensor cores' 128-byte swizzle, or 128 without.
bool delta_rows_map(CUtensorMap *m, const void *x, int64_t T, int H, int64_t stride, bool swizzle);

}  // namespace ra

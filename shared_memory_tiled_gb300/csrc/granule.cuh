// What an asynchronous copy takes of a bf16 row that is off 16-byte boundaries.
// For the device and, so that its addresses can be checked without a GPU, the host.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

namespace tr {

// Bytes between the 16-byte boundary at or below p and p.
__host__ __device__ __forceinline__ uint32_t granule_shift(const __nv_bfloat16 *p) {
    return uint32_t(reinterpret_cast<uintptr_t>(p) & 15u);
}

struct GranulePart {
    const __nv_bfloat16 *src;
    int bytes;
};

// The part of a 16-byte granule that lies in a row of `cols` values from `row` on; the
// granule begins at column col >= 0.  NULL where nothing of it does: a 16-byte copy
// wants a source on a 16-byte boundary however few bytes it takes, zero among
// them, and the row itself is off one.
__host__ __device__ __forceinline__ GranulePart granule_part(const __nv_bfloat16 *row, int64_t col, int64_t cols) {
    const int64_t left = cols - col;
    if (left <= 0) return GranulePart{nullptr, 0};
    return GranulePart{row + col, left < 8 ? int(left) * 2 : 16};
}

}  // namespace tr

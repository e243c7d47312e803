// Rounding to 8-bit floating point, as the quantizer and the norm's 8-bit output do it.
#pragma once

#include <cstdint>
#include <cuda_fp8.h>

#include "bounds.cuh"

namespace tr {

constexpr uint32_t kFloorBits = 0x0D800000u;  // 2^-100, the least block maximum that a scale is made from

// Eight values times r as eight bytes, the first lowest.
template <bool E5M2>
__device__ __forceinline__ uint2 to_bytes(const float (&v)[8], float r) {
    constexpr __nv_fp8_interpretation_t K = E5M2 ? __NV_E5M2 : __NV_E4M3;
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = __nv_cvt_float2_to_fp8x2(make_float2(v[2 * i] * r, v[2 * i + 1] * r), __NV_SATFINITE, K);
    return make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
}

// Eight bytes of one row at column c (a multiple of 8), those below `cols` only.
__device__ __forceinline__ void store8(uint8_t *row, int64_t c, int64_t cols, uint2 v,
                                       const dbg::Side &s) {
    if (c + 8 <= cols) {
        if (TR_STORE_OK(s, row + c, 8)) *reinterpret_cast<uint2 *>(row + c) = v;
        return;
    }
    for (int i = 0; i < 8 && c + i < cols; ++i)
        if (TR_STORE_OK(s, row + c + i, 1)) row[c + i] = uint8_t((i < 4 ? v.x >> (8 * i) : v.y >> (8 * (i - 4))));
}

}  // namespace tr

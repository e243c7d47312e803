// Rows of a matrix as 16-byte chunks: what the row-wise kernels (layer norm,
// its backward pass) share.
//
// A row that starts d elements past a 16-byte boundary is walked in chunks
// that do start on one: chunk c holds elements c*V - d .. c*V - d + V-1, the
// first and last of them partly outside the row.  Whole chunks move with one
// 16-byte access, the others element by element, so any base address and
// pitch reads and writes full sectors and never touches a byte outside the
// row.  A row's outputs line up with its chunks when they are offset alike.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "bounds.cuh"

namespace tr {

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) {
    return v;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
    return __float2bfloat16_rn(v);
}

template <typename T, int V>
struct alignas(V * sizeof(T)) Pack {
    T e[V];
};

// Elements between the 16-byte boundary at or below `row` and `row`.
template <typename T, int V>
__device__ __forceinline__ int row_shift(const T *row) {
    return V == 1 ? 0 : int((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T));
}

// Chunk with first element `lo` (may be negative) of a row of `cols`; elements
// outside the row read as zero.
template <typename T, int V>
__device__ __forceinline__ Pack<T, V> load_chunk(const T *row, int64_t lo, int64_t cols,
                                                 const dbg::Side &s) {
    Pack<T, V> p;
    if (lo >= 0 && lo + V <= cols) {
        if (TR_LOAD_OK(s, row + lo, int(sizeof(p)))) {
            if constexpr (sizeof(p) == 16) {
                const uint4 v = __ldcs(reinterpret_cast<const uint4 *>(row + lo));
                p = *reinterpret_cast<const Pack<T, V> *>(&v);
            } else {
                p = *reinterpret_cast<const Pack<T, V> *>(row + lo);
            }
            return p;
        }
    }
#pragma unroll
    for (int q = 0; q < V; ++q) {
        const bool in = lo + q >= 0 && lo + q < cols;
        p.e[q] = in && TR_LOAD_OK(s, row + lo + q, int(sizeof(T))) ? row[lo + q] : T(0.0f);
    }
    return p;
}

template <typename T, int V>
__device__ __forceinline__ void store_chunk(T *row, int64_t lo, int64_t cols, const Pack<T, V> &p,
                                            const dbg::Side &s) {
    if (lo >= 0 && lo + V <= cols) {
        if (TR_STORE_OK(s, row + lo, int(sizeof(p)))) {
            if constexpr (sizeof(p) == 16)
                __stcs(reinterpret_cast<uint4 *>(row + lo), *reinterpret_cast<const uint4 *>(&p));
            else
                *reinterpret_cast<Pack<T, V> *>(row + lo) = p;
        }
        return;
    }
#pragma unroll
    for (int q = 0; q < V; ++q)
        if (lo + q >= 0 && lo + q < cols && TR_STORE_OK(s, row + lo + q, int(sizeof(T))))
            row[lo + q] = p.e[q];
}

// Sum over the 32 lanes, in every lane.
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Sum over a group of TPR threads (32, or the whole block), in every thread;
// `slot` holds TPR/32 words.  Two calls in a row need two slots.
template <int TPR>
__device__ __forceinline__ float group_sum(float v, float *slot) {
    v = warp_sum(v);
    if constexpr (TPR > 32) {
        constexpr int NW = TPR / 32;
        const int lane = threadIdx.x & 31;
        if (lane == 0) slot[threadIdx.x >> 5] = v;
        __syncthreads();
        v = lane < NW ? slot[lane] : 0.0f;
        v = warp_sum(v);
    }
    return v;
}

// Weight j of a row of fp32 or bf16 weights.
__device__ __forceinline__ float weight(const void *w, bool w_bf16, int64_t j, const dbg::Side &s) {
    if (w_bf16) {
        const __nv_bfloat16 *p = static_cast<const __nv_bfloat16 *>(w) + j;
        return TR_LOAD_OK(s, p, 2) ? __bfloat162float(*p) : 0.0f;
    }
    const float *p = static_cast<const float *>(w) + j;
    return TR_LOAD_OK(s, p, 4) ? *p : 0.0f;
}

}  // namespace tr

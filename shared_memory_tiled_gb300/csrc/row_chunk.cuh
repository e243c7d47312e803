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
// The same, rounded to the type of the second argument; and a value stored in the type's way.
__device__ __forceinline__ float round_to(float v, float) { return v; }
__device__ __forceinline__ float round_to(float v, __nv_bfloat16) { return __bfloat162float(__float2bfloat16_rn(v)); }
__device__ __forceinline__ void put_value(float *p, float v) { *p = v; }
__device__ __forceinline__ void put_value(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

// V values of type T: 16 bytes, or one value.  bf16 stays packed in words.  A row in
// registers is unpacked once in every walk over it: the compiler would rather
// keep the first walk's unpacked values, twice the registers, and spill, so
// each walk after the first passes a zero that it cannot see through (`z`, one
// register per walk), which the byte permutation takes its zero bytes from.
template <typename T, int V>
struct Pack;

template <int V>
struct alignas(4 * V) Pack<float, V> {
    float e[V];
    __device__ __forceinline__ float get(int q) const { return e[q]; }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int q = 0; q < V; ++q) e[q] = 0.0f;
    }
    __device__ __forceinline__ void set(int q, float v) { e[q] = v; }
    __device__ __forceinline__ void round(const float (&v)[V]) {
#pragma unroll
        for (int q = 0; q < V; ++q) e[q] = v[q];
    }
    __device__ __forceinline__ float get(int q, uint32_t) const { return e[q]; }
};

template <>
struct alignas(16) Pack<__nv_bfloat16, 8> {
    uint32_t w[4];
    __device__ __forceinline__ float get(int q) const {
        return __uint_as_float(q & 1 ? w[q >> 1] & 0xffff0000u : w[q >> 1] << 16);
    }
    __device__ __forceinline__ void clear() { w[0] = w[1] = w[2] = w[3] = 0u; }
    // Into a cleared place.
    __device__ __forceinline__ void set(int q, __nv_bfloat16 v) {
        w[q >> 1] |= uint32_t(__bfloat16_as_ushort(v)) << (q & 1 ? 16 : 0);
    }
    __device__ __forceinline__ __nv_bfloat16 elem(int q) const {
        return __ushort_as_bfloat16(uint16_t(w[q >> 1] >> (q & 1 ? 16 : 0)));
    }
    __device__ __forceinline__ void round(const float (&v)[8]) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
            w[k] = *reinterpret_cast<const uint32_t *>(&h);
        }
    }
    __device__ __forceinline__ float get(int q, uint32_t z) const {
        return __uint_as_float(__byte_perm(w[q >> 1], z, q & 1 ? 0x3244 : 0x1044));
    }
};

template <>
struct Pack<__nv_bfloat16, 1> {
    __nv_bfloat16 e;
    __device__ __forceinline__ float get(int) const { return __bfloat162float(e); }
    __device__ __forceinline__ void clear() { e = __ushort_as_bfloat16(0); }
    __device__ __forceinline__ void set(int, __nv_bfloat16 v) { e = v; }
    __device__ __forceinline__ __nv_bfloat16 elem(int) const { return e; }
    __device__ __forceinline__ void round(const float (&v)[1]) { e = __float2bfloat16_rn(v[0]); }
    __device__ __forceinline__ float get(int q, uint32_t) const { return get(q); }
};

template <int V>
__device__ __forceinline__ float pack_elem(const Pack<float, V> &p, int q) {
    return p.e[q];
}
template <int V>
__device__ __forceinline__ __nv_bfloat16 pack_elem(const Pack<__nv_bfloat16, V> &p, int q) {
    return p.elem(q);
}

// Elements between the 16-byte boundary at or below `row` and `row`.
template <typename T, int V>
__device__ __forceinline__ int row_shift(const T *row) {
    return V == 1 ? 0 : int((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T));
}

// Chunk with first element `lo` (may be negative) of a row of `cols`; elements
// outside the row read as zero.  Without EDGE a chunk is whole or outside.
template <typename T, int V, bool EDGE = true>
__device__ __forceinline__ Pack<T, V> load_chunk(const T *row, int64_t lo, int64_t cols,
                                                 const dbg::Side &s) {
    Pack<T, V> p;
    if (lo >= 0 && lo + V <= cols && TR_LOAD_OK(s, row + lo, int(sizeof(p)))) {
        if constexpr (sizeof(p) == 16) {
            const uint4 v = __ldcs(reinterpret_cast<const uint4 *>(row + lo));
            p = *reinterpret_cast<const Pack<T, V> *>(&v);
        } else {
            p = *reinterpret_cast<const Pack<T, V> *>(row + lo);
        }
        return p;
    }
    p.clear();
    if constexpr (EDGE) {
#pragma unroll
        for (int q = 0; q < V; ++q)
            if (lo + q >= 0 && lo + q < cols && TR_LOAD_OK(s, row + lo + q, int(sizeof(T))))
                p.set(q, row[lo + q]);
    }
    return p;
}

template <typename T, int V, bool EDGE = true>
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
    if constexpr (EDGE) {
#pragma unroll
        for (int q = 0; q < V; ++q)
            if (lo + q >= 0 && lo + q < cols && TR_STORE_OK(s, row + lo + q, int(sizeof(T))))
                row[lo + q] = pack_elem(p, q);
    }
}

// Zeros for Pack::get: the launches here are one-dimensional.
__device__ __forceinline__ uint32_t opaque_zero_1() { return gridDim.y - 1; }
__device__ __forceinline__ uint32_t opaque_zero_2() { return gridDim.z - 1; }

// Sum over the 32 lanes, in every lane.
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Sums of R values over a group of TPR threads (32, or the whole block), in
// every thread; `slot` holds R * TPR/32 words.  Two calls in a row need two
// slots.
template <int TPR, int R>
__device__ __forceinline__ void group_sum(float (&v)[R], float *slot) {
#pragma unroll
    for (int r = 0; r < R; ++r) v[r] = warp_sum(v[r]);
    if constexpr (TPR > 32) {
        constexpr int NW = TPR / 32;
        const int lane = threadIdx.x & 31;
        if (lane == 0)
#pragma unroll
            for (int r = 0; r < R; ++r) slot[r * NW + (threadIdx.x >> 5)] = v[r];
        __syncthreads();
#pragma unroll
        for (int r = 0; r < R; ++r) v[r] = warp_sum(lane < NW ? slot[r * NW + lane] : 0.0f);
    }
}

// V weights from `lo` on (a whole chunk on a 16-byte boundary).
template <int V>
__device__ __forceinline__ void load_weights(const void *w, bool w_bf16, int64_t lo, float (&v)[V],
                                             const dbg::Side &s) {
    if (w_bf16) {
        const __nv_bfloat16 *p = static_cast<const __nv_bfloat16 *>(w) + lo;
#pragma unroll
        for (int q = 0; q < V; q += 4) {
            uint2 b = make_uint2(0u, 0u);
            if (TR_LOAD_OK(s, p + q, 8)) b = *reinterpret_cast<const uint2 *>(p + q);
            v[q] = __uint_as_float(b.x << 16);
            v[q + 1] = __uint_as_float(b.x & 0xffff0000u);
            v[q + 2] = __uint_as_float(b.y << 16);
            v[q + 3] = __uint_as_float(b.y & 0xffff0000u);
        }
    } else {
        const float *p = static_cast<const float *>(w) + lo;
#pragma unroll
        for (int q = 0; q < V; q += 4) {
            float4 f = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (TR_LOAD_OK(s, p + q, 16)) f = *reinterpret_cast<const float4 *>(p + q);
            v[q] = f.x;
            v[q + 1] = f.y;
            v[q + 2] = f.z;
            v[q + 3] = f.w;
        }
    }
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

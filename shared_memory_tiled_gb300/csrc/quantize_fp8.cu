// Quantizing to 8-bit floating point with a scale for each block of 128, row
// by row and transposed from one read.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "bounds.cuh"
#include "launch.cuh"
#include "tr_internal.h"

namespace tr {
namespace {

constexpr int kThreads = 256;
constexpr uint32_t kFloorBits = 0x0D800000u;  // 2^-100

struct Quant {
    const void *x;
    uint8_t *q, *qt;
    float *scale, *scale_t;
    int64_t rows, cols, ld_x, ld_q, ld_scale, ld_qt, ld_scale_t;
    int64_t tiles_r, tiles_c;
    float top;  // the 8-bit type's largest finite value
};

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

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

// One 128 x 128 tile per turn.  A thread holds the 8 x 8 values of row group rg
// and column group cg; 16 lanes share a row group, so a row's maximum is a
// shuffle and a column's goes through shared memory.  Row bytes are stored
// straight from the registers (16 lanes write 128 contiguous bytes); the
// transposed ones go through a shared tile of 8-byte slots, slot XOR column
// group, so that neither its writes nor its reads share a bank.
template <typename T, bool VEC, bool E5M2, bool BLOCK, bool BOTH>
__global__ void __launch_bounds__(kThreads) k_quantize(Quant a) {
    pdl_prologue();
    __shared__ uint32_t col_max[8][128];
    __shared__ uint2 turned[BOTH ? 128 * 16 : 1];
    [[maybe_unused]] const dbg::Side sx = dbg::side(a.x, 1, a.rows, a.cols, a.ld_x, 0, sizeof(T));
    [[maybe_unused]] const dbg::Side sq = dbg::side(a.q, 1, a.rows, a.cols, a.ld_q, 0, 1);
    [[maybe_unused]] const dbg::Side st = dbg::side(a.qt, 1, a.cols, a.rows, a.ld_qt, 0, 1);
    [[maybe_unused]] const dbg::Side ss = dbg::side(a.scale, 1, a.tiles_c, BLOCK ? a.tiles_r : a.rows, a.ld_scale, 0, 4);
    [[maybe_unused]] const dbg::Side su = dbg::side(a.scale_t, 1, a.tiles_r, BLOCK ? a.tiles_c : a.cols, a.ld_scale_t, 0, 4);
    const int t = threadIdx.x, cg = t & 15, rg = t >> 4, warp = t >> 5;
    const T *x = static_cast<const T *>(a.x);
    for (int64_t tile = blockIdx.x; tile < a.tiles_r * a.tiles_c; tile += gridDim.x) {
        const int64_t tr = tile / a.tiles_c, tc = tile - tr * a.tiles_c;
        const int64_t r0 = tr * 128 + rg * 8, c0 = tc * 128 + cg * 8;
        float v[8][8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const T *p = x + (r0 + i) * a.ld_x + c0;
            if (VEC && r0 + i < a.rows && c0 + 8 <= a.cols && TR_LOAD_OK(sx, p, int(8 * sizeof(T)))) {
                constexpr int N = int(sizeof(T)) / 2;
                uint4 raw[N];
#pragma unroll
                for (int k = 0; k < N; ++k) raw[k] = __ldcs(reinterpret_cast<const uint4 *>(p) + k);
                const T *e = reinterpret_cast<const T *>(raw);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] = float(e[j]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    v[i][j] = r0 + i < a.rows && c0 + j < a.cols && TR_LOAD_OK(sx, p + j, int(sizeof(T)))
                                  ? float(p[j]) : 0.0f;
            }
        }
        uint32_t rm[8], cm[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            rm[i] = kFloorBits;
            cm[i] = kFloorBits;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t b = abs_bits(v[i][j]);
                rm[i] = max(rm[i], b);
                cm[j] = max(cm[j], b);
            }
        if constexpr (BLOCK) {
            uint32_t m = kFloorBits;
#pragma unroll
            for (int i = 0; i < 8; ++i) m = max(m, rm[i]);
            m = __reduce_max_sync(0xffffffffu, m);
            if ((t & 31) == 0) col_max[0][warp] = m;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < 8; ++w) m = max(m, col_max[0][w]);
#pragma unroll
            for (int i = 0; i < 8; ++i) rm[i] = cm[i] = m;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int o = 8; o; o >>= 1) rm[i] = max(rm[i], __shfl_xor_sync(0xffffffffu, rm[i], o));
            if constexpr (BOTH) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    cm[j] = max(cm[j], __shfl_xor_sync(0xffffffffu, cm[j], 16));
                    if ((t & 16) == 0) col_max[warp][cg * 8 + j] = cm[j];
                }
                __syncthreads();
#pragma unroll
                for (int j = 0; j < 8; ++j)
#pragma unroll
                    for (int w = 0; w < 8; ++w) cm[j] = max(cm[j], col_max[w][cg * 8 + j]);
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (r0 + i >= a.rows) continue;
            const float m = __uint_as_float(rm[i]);
            store8(a.q + (r0 + i) * a.ld_q, c0, a.cols, to_bytes<E5M2>(v[i], a.top / m), sq);
            if (BLOCK ? t == 0 && i == 0 : cg == 0) {
                float *s = a.scale + tc * a.ld_scale + (BLOCK ? tr : r0 + i);
                if (TR_STORE_OK(ss, s, 4)) *s = m / a.top;
            }
        }
        if constexpr (BOTH) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float m = __uint_as_float(cm[j]);
                float col[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) col[i] = v[i][j];
                turned[(cg * 8 + j) * 16 + (rg ^ cg)] = to_bytes<E5M2>(col, a.top / m);
                if ((BLOCK ? t == 0 && j == 0 : rg == 0) && c0 + j < a.cols) {
                    float *s = a.scale_t + tr * a.ld_scale_t + (BLOCK ? tc : c0 + j);
                    if (TR_STORE_OK(su, s, 4)) *s = m / a.top;
                }
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int c = i * 16 + rg;
                const int64_t col = tc * 128 + c;
                if (col < a.cols)
                    store8(a.qt + col * a.ld_qt, tr * 128 + cg * 8, a.rows, turned[c * 16 + (cg ^ (c >> 3))], st);
            }
        }
        if (BOTH || BLOCK) __syncthreads();  // the shared words are written anew in the next turn
    }
}

template <typename T, bool VEC, bool E5M2>
cudaError_t launch_typed(const Quant &a, bool block, cudaStream_t stream) {
    const int64_t tiles = a.tiles_r * a.tiles_c, most = int64_t(1) << 30;
    const dim3 grid(unsigned(tiles < most ? tiles : most)), threads(kThreads);
    if (block)
        return a.qt ? launch_pdl(k_quantize<T, VEC, E5M2, true, true>, grid, threads, 0, stream, a)
                    : launch_pdl(k_quantize<T, VEC, E5M2, true, false>, grid, threads, 0, stream, a);
    return a.qt ? launch_pdl(k_quantize<T, VEC, E5M2, false, true>, grid, threads, 0, stream, a)
                : launch_pdl(k_quantize<T, VEC, E5M2, false, false>, grid, threads, 0, stream, a);
}

template <typename T>
cudaError_t launch_in(const Quant &a, bool block, bool e5m2, cudaStream_t stream) {
    const bool vec = side_aligned16(a.x, a.ld_x, 0, 1, sizeof(T));
    if (vec) return e5m2 ? launch_typed<T, true, true>(a, block, stream) : launch_typed<T, true, false>(a, block, stream);
    return e5m2 ? launch_typed<T, false, true>(a, block, stream) : launch_typed<T, false, false>(a, block, stream);
}

}  // namespace

// Debug builds: this unit's record of refused accesses.
TR_BOUNDS_READER(read_bounds_quantize)

cudaError_t launch_quantize(const tr_quantize_args &p) {
    const bool e5m2 = p.q_dtype == TR_DTYPE_E5M2;
    const Quant a{p.x, static_cast<uint8_t *>(p.q), static_cast<uint8_t *>(p.qt), p.scale, p.scale_t,
                  p.rows, p.cols, p.ld_x, p.ld_q, p.ld_scale, p.ld_qt, p.ld_scale_t,
                  (p.rows + 127) / 128, (p.cols + 127) / 128, e5m2 ? 57344.0f : 448.0f};
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(p.stream);
    return p.x_dtype == TR_DTYPE_F32 ? launch_in<float>(a, p.block_rows == 128, e5m2, stream)
                                     : launch_in<__nv_bfloat16>(a, p.block_rows == 128, e5m2, stream);
}

}  // namespace tr

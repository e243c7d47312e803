// Root-mean-square norm with the residual's addition: h = x + residual, and
// y = h * rstd * gamma with rstd = 1 / sqrt(sum(h^2) / n + eps), as rows of h's type and in
// 8 bits with a scale for each block of 128, by rows and transposed.
//
// Bound by memory: x and residual are read once, h, y, q and qt written once.
#include "fp8.cuh"
#include "launch.cuh"
#include "row_chunk.cuh"
#include "tr_internal.h"

namespace tr {
namespace {

struct Rms {
    const void *x, *residual, *gamma;
    void *h, *y;
    float *rstd;
    uint8_t *q, *qt;
    float *scale, *scale_t;
    int64_t rows, cols, ld_x, ld_residual, ld_h, ld_y, ld_q, ld_scale, ld_qt, ld_scale_t;
    float eps, inv_cols, top;
    bool w_bf16, e5m2;
};

__device__ __forceinline__ uint8_t to_byte(float v, bool e5m2) {
    return __nv_cvt_float_to_fp8(v, __NV_SATFINITE, e5m2 ? __NV_E5M2 : __NV_E4M3);
}

// One row to a block, in two walks, one value to an access.
template <typename T>
__global__ void __launch_bounds__(1024) k_rmsnorm_any(const Rms a) {
    pdl_prologue();
    __shared__ float slots[2][32];
    [[maybe_unused]] const dbg::Side sx = dbg::side(a.x, 1, a.rows, a.cols, a.ld_x, 0, sizeof(T));
    [[maybe_unused]] const dbg::Side sr = dbg::side(a.residual, 1, a.rows, a.cols, a.ld_residual, 0, sizeof(T));
    [[maybe_unused]] const dbg::Side sh = dbg::side(a.h, 1, a.rows, a.cols, a.ld_h, 0, sizeof(T));
    [[maybe_unused]] const dbg::Side sy = dbg::side(a.y, 1, a.rows, a.cols, a.ld_y, 0, sizeof(T));
    [[maybe_unused]] const dbg::Side sw = dbg::side(a.gamma, 1, 1, a.cols, a.cols, 0, a.w_bf16 ? 2 : 4);
    [[maybe_unused]] const dbg::Side sd = dbg::side(a.rstd, 1, 1, a.rows, a.rows, 0, 4);
    [[maybe_unused]] const dbg::Side sq = dbg::side(a.q, 1, a.rows, a.cols, a.ld_q, 0, 1);
    [[maybe_unused]] const dbg::Side ss = dbg::side(a.scale, 1, (a.cols + 127) / 128, a.rows, a.ld_scale, 0, 4);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int turn = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
        const T *x = static_cast<const T *>(a.x) + row * a.ld_x;
        const T *r = static_cast<const T *>(a.residual) + row * a.ld_residual;
        T *h = static_cast<T *>(a.h) + row * a.ld_h;
        T *y = static_cast<T *>(a.y) + row * a.ld_y;
        float sum[1] = {0.0f};
        for (int64_t j = threadIdx.x; j < a.cols; j += blockDim.x) {
            float v = TR_LOAD_OK(sx, x + j, int(sizeof(T))) ? to_f32(x[j]) : 0.0f;
            if (a.residual) {
                if (TR_LOAD_OK(sr, r + j, int(sizeof(T)))) v += to_f32(r[j]);
                v = round_to(v, T(0.0f));
                if (TR_STORE_OK(sh, h + j, int(sizeof(T)))) put_value(h + j, v);
            }
            sum[0] = fmaf(v, v, sum[0]);
        }
        group_sum<1024, 1>(sum, slots[turn]);
        const float rstd = 1.0f / sqrtf(fmaf(sum[0], a.inv_cols, a.eps));
        if (threadIdx.x == 0 && a.rstd && TR_STORE_OK(sd, a.rstd + row, 4)) a.rstd[row] = rstd;
        const T *from = a.residual ? h : x;
        for (int64_t c0 = int64_t(warp) * 128; c0 < a.cols; c0 += int64_t(blockDim.x) * 4) {
            float v[4];
            uint32_t most = kFloorBits;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int64_t j = c0 + k * 32 + lane;
                v[k] = j < a.cols ? to_f32(from[j]) * rstd * weight(a.gamma, a.w_bf16, j, sw) : 0.0f;
                if (a.y && j < a.cols && TR_STORE_OK(sy, y + j, int(sizeof(T)))) put_value(y + j, v[k]);
                most = max(most, __float_as_uint(v[k]) & 0x7fffffffu);
            }
            if (!a.q) continue;
            const float amax = __uint_as_float(__reduce_max_sync(0xffffffffu, most));
            const float inv = a.top / amax;
            if (lane == 0) {
                float *s = a.scale + (c0 >> 7) * a.ld_scale + row;
                if (TR_STORE_OK(ss, s, 4)) *s = amax / a.top;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int64_t j = c0 + k * 32 + lane;
                uint8_t *q = a.q + row * a.ld_q + j;
                if (j < a.cols && TR_STORE_OK(sq, q, 1)) *q = to_byte(v[k] * inv, a.e5m2);
            }
        }
    }
}

// The transposed 8-bit output of a 128 x 128 tile, from h and rstd: a thread walks half a column
// twice, and the bytes go through shared memory.
template <typename T>
__global__ void __launch_bounds__(256) k_rmsnorm_turned(const Rms a) {
    pdl_prologue();
    __shared__ uint32_t col_max[2][128];
    __shared__ uint8_t tile[128][132];
    const void *src = a.residual ? a.h : a.x;
    const int64_t ld = a.residual ? a.ld_h : a.ld_x;
    [[maybe_unused]] const dbg::Side sh = dbg::side(src, 1, a.rows, a.cols, ld, 0, sizeof(T));
    [[maybe_unused]] const dbg::Side sw = dbg::side(a.gamma, 1, 1, a.cols, a.cols, 0, a.w_bf16 ? 2 : 4);
    [[maybe_unused]] const dbg::Side sd = dbg::side(a.rstd, 1, 1, a.rows, a.rows, 0, 4);
    [[maybe_unused]] const dbg::Side st = dbg::side(a.qt, 1, a.cols, a.rows, a.ld_qt, 0, 1);
    [[maybe_unused]] const dbg::Side su = dbg::side(a.scale_t, 1, (a.rows + 127) / 128, a.cols, a.ld_scale_t, 0, 4);
    const int64_t tiles_r = (a.rows + 127) / 128, tiles_c = (a.cols + 127) / 128;
    const int c = threadIdx.x & 127, half = threadIdx.x >> 7;
    for (int64_t at = blockIdx.x; at < tiles_r * tiles_c; at += gridDim.x) {
        const int64_t r0 = at / tiles_c * 128, c0 = at % tiles_c * 128, col = c0 + c;
        const float w = col < a.cols ? weight(a.gamma, a.w_bf16, col, sw) : 0.0f;
        auto value = [&](int i) {
            const int64_t row = r0 + half * 64 + i;
            if (row >= a.rows || col >= a.cols) return 0.0f;
            const T *p = static_cast<const T *>(src) + row * ld + col;
            return TR_LOAD_OK(sh, p, int(sizeof(T))) && TR_LOAD_OK(sd, a.rstd + row, 4) ? to_f32(*p) * a.rstd[row] * w : 0.0f;
        };
        uint32_t most = kFloorBits;
        for (int i = 0; i < 64; ++i) most = max(most, __float_as_uint(value(i)) & 0x7fffffffu);
        col_max[half][c] = most;
        __syncthreads();
        const float amax = __uint_as_float(max(col_max[0][c], col_max[1][c])), inv = a.top / amax;
        if (half == 0 && col < a.cols) {
            float *s = a.scale_t + (r0 >> 7) * a.ld_scale_t + col;
            if (TR_STORE_OK(su, s, 4)) *s = amax / a.top;
        }
        for (int i = 0; i < 64; ++i) tile[c][half * 64 + i] = to_byte(value(i) * inv, a.e5m2);
        __syncthreads();
        for (int k = threadIdx.x; k < 128 * 128; k += 256) {
            const int64_t j = c0 + (k >> 7), row = r0 + (k & 127);
            uint8_t *p = a.qt + j * a.ld_qt + row;
            if (j < a.cols && row < a.rows && TR_STORE_OK(st, p, 1)) *p = tile[k >> 7][k & 127];
        }
        __syncthreads();
    }
}

template <typename T>
cudaError_t launch_typed(const Rms &a, cudaStream_t stream) {
    const int64_t most = int64_t(1) << 30;
    cudaError_t e = launch_pdl(k_rmsnorm_any<T>, dim3(unsigned(a.rows < most ? a.rows : most)), dim3(1024), 0, stream, a);
    if (e != cudaSuccess || !a.qt) return e;
    const int64_t tiles = ((a.rows + 127) / 128) * ((a.cols + 127) / 128);
    return launch_pdl(k_rmsnorm_turned<T>, dim3(unsigned(tiles < most ? tiles : most)), dim3(256), 0, stream, a);
}

}  // namespace

// Debug builds: this unit's record of refused accesses.
TR_BOUNDS_READER(read_bounds_rmsnorm)

cudaError_t launch_rmsnorm(const tr_rmsnorm_args &p) {
    const bool e5m2 = p.q_dtype == TR_DTYPE_E5M2;
    const Rms a{p.x, p.residual, p.gamma, p.h, p.y, p.rstd, static_cast<uint8_t *>(p.q), static_cast<uint8_t *>(p.qt), p.scale, p.scale_t,
                p.rows, p.cols, p.ld_x, p.ld_residual, p.ld_h, p.ld_y, p.ld_q, p.ld_scale, p.ld_qt, p.ld_scale_t,
                p.eps, 1.0f / float(p.cols), e5m2 ? 57344.0f : 448.0f, p.w_dtype == TR_DTYPE_BF16, e5m2};
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(p.stream);
    return p.x_dtype == TR_DTYPE_F32 ? launch_typed<float>(a, stream) : launch_typed<__nv_bfloat16>(a, stream);
}

}  // namespace tr

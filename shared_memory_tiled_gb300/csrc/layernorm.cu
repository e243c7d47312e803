// Layer norm, forward: y = (x - mean) * rstd * gamma + beta along each row.
#include "launch.cuh"
#include "row_chunk.cuh"
#include "tr_internal.h"

namespace tr {
namespace {

// TPR threads hold one row, NCH chunks each, in registers: x is read once and
// the deviations are summed about the mean from the registers.
template <typename T, int V, int TPR, int NCH>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR)
k_layernorm(const T *__restrict__ x, const void *__restrict__ gamma, const void *__restrict__ beta,
            T *__restrict__ y, float *__restrict__ mean_out, float *__restrict__ rstd_out,
            int64_t rows, int64_t cols, int64_t ld_x, int64_t ld_y, float eps, bool w_bf16) {
    pdl_prologue();
    constexpr int RPB = (TPR < 128 ? 128 : TPR) / TPR;
    __shared__ float slots[2][32];
    [[maybe_unused]] const dbg::Side sx = dbg::side(x, 1, rows, cols, ld_x, 0, sizeof(T));
    [[maybe_unused]] const dbg::Side sy = dbg::side(y, 1, rows, cols, ld_y, 0, sizeof(T));
    [[maybe_unused]] const dbg::Side sw = dbg::side(gamma, 1, 1, cols, cols, 0, w_bf16 ? 2 : 4);
    [[maybe_unused]] const dbg::Side sb = dbg::side(beta, 1, 1, cols, cols, 0, w_bf16 ? 2 : 4);
    [[maybe_unused]] const dbg::Side ss = dbg::side(mean_out, 1, 1, rows, rows, 0, 4);
    [[maybe_unused]] const dbg::Side sr = dbg::side(rstd_out, 1, 1, rows, rows, 0, 4);
    const int t = threadIdx.x % TPR;
    const float inv_cols = 1.0f / float(cols);
    for (int64_t row = int64_t(blockIdx.x) * RPB + threadIdx.x / TPR; row < rows;
         row += int64_t(gridDim.x) * RPB) {
        const T *xr = x + row * ld_x;
        const int d = row_shift<T, V>(xr);
        Pack<T, V> p[NCH];
#pragma unroll
        for (int i = 0; i < NCH; ++i)
            p[i] = load_chunk<T, V>(xr, int64_t(t + i * TPR) * V - d, cols, sx);
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < NCH; ++i)
#pragma unroll
            for (int q = 0; q < V; ++q) sum += to_f32(p[i].e[q]);
        const float mean = group_sum<TPR>(sum, slots[0]) * inv_cols;
        float dev = 0.0f;
#pragma unroll
        for (int i = 0; i < NCH; ++i)
#pragma unroll
            for (int q = 0; q < V; ++q) {
                const int64_t j = int64_t(t + i * TPR) * V - d + q;
                const float o = to_f32(p[i].e[q]) - mean;
                if (j >= 0 && j < cols) dev = fmaf(o, o, dev);
            }
        const float var = group_sum<TPR>(dev, slots[1]) * inv_cols;
        const float rstd = 1.0f / sqrtf(var + eps);
        T *yr = y + row * ld_y;
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const int64_t lo = int64_t(t + i * TPR) * V - d;
            if (lo >= cols) continue;
            Pack<T, V> o;
#pragma unroll
            for (int q = 0; q < V; ++q) {
                const int64_t j = lo + q;
                if (j < 0 || j >= cols) continue;
                float v = (to_f32(p[i].e[q]) - mean) * rstd * weight(gamma, w_bf16, j, sw);
                if (beta) v += weight(beta, w_bf16, j, sb);
                o.e[q] = from_f32<T>(v);
            }
            store_chunk<T, V>(yr, lo, cols, o, sy);
        }
        if (t == 0) {
            if (mean_out && TR_STORE_OK(ss, mean_out + row, 4)) mean_out[row] = mean;
            if (rstd_out && TR_STORE_OK(sr, rstd_out + row, 4)) rstd_out[row] = rstd;
        }
    }
}

// Rows too long for registers, and rows whose x and y are offset differently
// from a 16-byte boundary (V = 1): a block walks its row three times.
template <typename T, int V>
__global__ void __launch_bounds__(1024)
k_layernorm_long(const T *__restrict__ x, const void *__restrict__ gamma,
                 const void *__restrict__ beta, T *__restrict__ y, float *__restrict__ mean_out,
                 float *__restrict__ rstd_out, int64_t rows, int64_t cols, int64_t ld_x,
                 int64_t ld_y, float eps, bool w_bf16) {
    pdl_prologue();
    __shared__ float slots[2][32];
    [[maybe_unused]] const dbg::Side sx = dbg::side(x, 1, rows, cols, ld_x, 0, sizeof(T));
    [[maybe_unused]] const dbg::Side sy = dbg::side(y, 1, rows, cols, ld_y, 0, sizeof(T));
    [[maybe_unused]] const dbg::Side sw = dbg::side(gamma, 1, 1, cols, cols, 0, w_bf16 ? 2 : 4);
    [[maybe_unused]] const dbg::Side sb = dbg::side(beta, 1, 1, cols, cols, 0, w_bf16 ? 2 : 4);
    [[maybe_unused]] const dbg::Side ss = dbg::side(mean_out, 1, 1, rows, rows, 0, 4);
    [[maybe_unused]] const dbg::Side sr = dbg::side(rstd_out, 1, 1, rows, rows, 0, 4);
    const float inv_cols = 1.0f / float(cols);
    const int64_t step = int64_t(blockDim.x) * V;
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
        const T *xr = x + row * ld_x;
        const int d = row_shift<T, V>(xr);
        const int64_t first = int64_t(threadIdx.x) * V - d;
        float sum = 0.0f;
        for (int64_t lo = first; lo < cols; lo += step) {
            const Pack<T, V> p = load_chunk<T, V>(xr, lo, cols, sx);
#pragma unroll
            for (int q = 0; q < V; ++q) sum += to_f32(p.e[q]);
        }
        const float mean = group_sum<1024>(sum, slots[0]) * inv_cols;
        float dev = 0.0f;
        for (int64_t lo = first; lo < cols; lo += step) {
            const Pack<T, V> p = load_chunk<T, V>(xr, lo, cols, sx);
#pragma unroll
            for (int q = 0; q < V; ++q) {
                const float o = to_f32(p.e[q]) - mean;
                if (lo + q >= 0 && lo + q < cols) dev = fmaf(o, o, dev);
            }
        }
        const float var = group_sum<1024>(dev, slots[1]) * inv_cols;
        const float rstd = 1.0f / sqrtf(var + eps);
        T *yr = y + row * ld_y;
        for (int64_t lo = first; lo < cols; lo += step) {
            Pack<T, V> p = load_chunk<T, V>(xr, lo, cols, sx);
#pragma unroll
            for (int q = 0; q < V; ++q) {
                const int64_t j = lo + q;
                if (j < 0 || j >= cols) continue;
                float v = (to_f32(p.e[q]) - mean) * rstd * weight(gamma, w_bf16, j, sw);
                if (beta) v += weight(beta, w_bf16, j, sb);
                p.e[q] = from_f32<T>(v);
            }
            store_chunk<T, V>(yr, lo, cols, p, sy);
        }
        if (threadIdx.x == 0) {
            if (mean_out && TR_STORE_OK(ss, mean_out + row, 4)) mean_out[row] = mean;
            if (rstd_out && TR_STORE_OK(sr, rstd_out + row, 4)) rstd_out[row] = rstd;
        }
    }
}

template <typename T>
cudaError_t launch_typed(const tr_layernorm_args &a) {
    constexpr int V = 16 / int(sizeof(T));
    const T *x = static_cast<const T *>(a.x);
    T *y = static_cast<T *>(a.y);
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(a.stream);
    const bool w_bf16 = a.w_dtype == TR_DTYPE_BF16;
    const int64_t most = int64_t(1) << 30;
    auto run = [&](auto kern, int threads, int rows_per_block) {
        int64_t grid = (a.rows + rows_per_block - 1) / rows_per_block;
        if (grid > most) grid = most;
        return launch_pdl(kern, dim3(unsigned(grid)), dim3(threads), 0, stream, x, a.gamma, a.beta,
                          y, a.mean, a.rstd, a.rows, a.cols, a.ld_x, a.ld_y, a.eps, w_bf16);
    };
    const uintptr_t ax = reinterpret_cast<uintptr_t>(x), ay = reinterpret_cast<uintptr_t>(y);
    const bool alike = ((ax ^ ay) & 15u) == 0 && ((a.ld_x - a.ld_y) * int64_t(sizeof(T))) % 16 == 0;
    if (!alike) return run(k_layernorm_long<T, 1>, 1024, 1);
    const bool shifted = (ax & 15u) != 0 || (a.ld_x * int64_t(sizeof(T))) % 16 != 0;
    const int64_t chunks = (a.cols + (shifted ? V - 1 : 0) + V - 1) / V;
    if (chunks <= 32) return run(k_layernorm<T, V, 32, 1>, 128, 4);
    if (chunks <= 64) return run(k_layernorm<T, V, 32, 2>, 128, 4);
    if (chunks <= 128) return run(k_layernorm<T, V, 32, 4>, 128, 4);
    if (chunks <= 256) return run(k_layernorm<T, V, 128, 2>, 128, 1);
    if (chunks <= 512) return run(k_layernorm<T, V, 128, 4>, 128, 1);
    if (chunks <= 1024) return run(k_layernorm<T, V, 256, 4>, 256, 1);
    if (chunks <= 2048) return run(k_layernorm<T, V, 512, 4>, 512, 1);
    if (chunks <= 4096) return run(k_layernorm<T, V, 512, 8>, 512, 1);
    return run(k_layernorm_long<T, V>, 1024, 1);
}

}  // namespace

// Debug builds: this unit's record of refused accesses.
TR_BOUNDS_READER(read_bounds_layernorm)

cudaError_t launch_layernorm(const tr_layernorm_args &a) {
    return a.x_dtype == TR_DTYPE_F32 ? launch_typed<float>(a) : launch_typed<__nv_bfloat16>(a);
}

}  // namespace tr

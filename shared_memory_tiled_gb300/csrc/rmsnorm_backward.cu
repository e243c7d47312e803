// Root-mean-square norm, backward: the gradient of what was normed along the rows, the
// weight's down the columns.  With u = h * rstd and g = dy * gamma,
//
//   dx = rstd * (g - u * sum(g u)/n) + dresidual,  dgamma = sum_rows dy u
//
// Bound by memory: one read of dy, h and dresidual, one write of dx.
#include "launch.cuh"
#include "row_chunk.cuh"
#include "tr_internal.h"

namespace tr {
namespace {

struct RmsBwd {
    const void *dy, *h, *gamma;
    const float *rstd;
    const void *dres;
    void *dx;
    float *dgamma, *part;
    int64_t rows, cols, ld_dy, ld_h, ld_dres, ld_dx;
    int64_t parts, rows_per_part;
    bool w_bf16;
};

// dx of one row per block, in two walks along it.
template <typename T>
__global__ void __launch_bounds__(512) k_rms_dx(const RmsBwd a) {
    pdl_prologue();
    __shared__ float slots[2][16];
    [[maybe_unused]] const dbg::Side sd = dbg::side(a.dy, 1, a.rows, a.cols, a.ld_dy, 0, sizeof(T));
    [[maybe_unused]] const dbg::Side sh = dbg::side(a.h, 1, a.rows, a.cols, a.ld_h, 0, sizeof(T));
    [[maybe_unused]] const dbg::Side se = dbg::side(a.dres, 1, a.rows, a.cols, a.ld_dres, 0, sizeof(T));
    [[maybe_unused]] const dbg::Side so = dbg::side(a.dx, 1, a.rows, a.cols, a.ld_dx, 0, sizeof(T));
    [[maybe_unused]] const dbg::Side sw = dbg::side(a.gamma, 1, 1, a.cols, a.cols, 0, a.w_bf16 ? 2 : 4);
    [[maybe_unused]] const dbg::Side sr = dbg::side(a.rstd, 1, 1, a.rows, a.rows, 0, 4);
    const float inv_cols = 1.0f / float(a.cols);
    int turn = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
        const T *dy = static_cast<const T *>(a.dy) + row * a.ld_dy;
        const T *h = static_cast<const T *>(a.h) + row * a.ld_h;
        const T *dr = static_cast<const T *>(a.dres) + row * a.ld_dres;
        T *dx = static_cast<T *>(a.dx) + row * a.ld_dx;
        const float rstd = TR_LOAD_OK(sr, a.rstd + row, 4) ? a.rstd[row] : 0.0f;
        float s[1] = {0.0f};
        for (int64_t j = threadIdx.x; j < a.cols; j += blockDim.x) {
            if (!TR_LOAD_OK(sd, dy + j, int(sizeof(T))) || !TR_LOAD_OK(sh, h + j, int(sizeof(T)))) continue;
            s[0] = fmaf(to_f32(dy[j]) * weight(a.gamma, a.w_bf16, j, sw), to_f32(h[j]) * rstd, s[0]);
        }
        group_sum<512, 1>(s, slots[turn]);
        const float c = s[0] * inv_cols;
        for (int64_t j = threadIdx.x; j < a.cols; j += blockDim.x) {
            if (!TR_LOAD_OK(sd, dy + j, int(sizeof(T))) || !TR_LOAD_OK(sh, h + j, int(sizeof(T)))) continue;
            const float g = to_f32(dy[j]) * weight(a.gamma, a.w_bf16, j, sw), u = to_f32(h[j]) * rstd;
            float v = rstd * fmaf(-u, c, g);
            if (a.dres && TR_LOAD_OK(se, dr + j, int(sizeof(T)))) v += to_f32(dr[j]);
            if (TR_STORE_OK(so, dx + j, int(sizeof(T)))) put_value(dx + j, v);
        }
    }
}

// Column sums of dy*u over one part of the rows: 32 columns by 8 rows of threads.
template <typename T>
__global__ void __launch_bounds__(256) k_rms_columns(const RmsBwd a) {
    pdl_prologue();
    __shared__ float red[8][33];
    [[maybe_unused]] const dbg::Side sd = dbg::side(a.dy, 1, a.rows, a.cols, a.ld_dy, 0, sizeof(T));
    [[maybe_unused]] const dbg::Side sh = dbg::side(a.h, 1, a.rows, a.cols, a.ld_h, 0, sizeof(T));
    [[maybe_unused]] const dbg::Side sp = dbg::side(a.part, 1, a.parts, a.cols, a.cols, 0, 4);
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int64_t part = blockIdx.y;
    const int64_t r0 = part * a.rows_per_part;
    const int64_t r1 = r0 + a.rows_per_part < a.rows ? r0 + a.rows_per_part : a.rows;
    for (int64_t c0 = int64_t(blockIdx.x) * 32; c0 < a.cols; c0 += int64_t(gridDim.x) * 32) {
        const int64_t j = c0 + tx;
        float s = 0.0f;
        if (j < a.cols)
            for (int64_t r = r0 + ty; r < r1; r += 8) {
                const T *pd = static_cast<const T *>(a.dy) + r * a.ld_dy + j;
                const T *ph = static_cast<const T *>(a.h) + r * a.ld_h + j;
                if (!TR_LOAD_OK(sd, pd, int(sizeof(T))) || !TR_LOAD_OK(sh, ph, int(sizeof(T)))) continue;
                s = fmaf(to_f32(*pd), to_f32(*ph) * a.rstd[r], s);
            }
        red[ty][tx] = s;
        __syncthreads();
        if (ty == 0 && j < a.cols) {
#pragma unroll
            for (int i = 1; i < 8; ++i) s += red[i][tx];
            float *p = a.part + part * a.cols + j;
            if (TR_STORE_OK(sp, p, 4)) *p = s;
        }
        __syncthreads();
    }
}

// The parts' sums: 32 columns by 8 rows of threads, each over every eighth part,
// joined in a fixed order.
__global__ void __launch_bounds__(256) k_rms_join(const RmsBwd a) {
    pdl_prologue();
    __shared__ float red[8][33];
    [[maybe_unused]] const dbg::Side sp = dbg::side(a.part, 1, a.parts, a.cols, a.cols, 0, 4);
    [[maybe_unused]] const dbg::Side so = dbg::side(a.dgamma, 1, 1, a.cols, a.cols, 0, 4);
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    for (int64_t c0 = int64_t(blockIdx.x) * 32; c0 < a.cols; c0 += int64_t(gridDim.x) * 32) {
        const int64_t j = c0 + tx;
        float s = 0.0f;
        if (j < a.cols)
#pragma unroll 8
            for (int64_t i = ty; i < a.parts; i += 8) {
                const float *p = a.part + i * a.cols + j;
                if (TR_LOAD_OK(sp, p, 4)) s += *p;
            }
        red[ty][tx] = s;
        __syncthreads();
        if (ty == 0 && j < a.cols) {
#pragma unroll
            for (int k = 1; k < 8; ++k) s += red[k][tx];
            if (TR_STORE_OK(so, a.dgamma + j, 4)) a.dgamma[j] = s;
        }
        __syncthreads();
    }
}

// Most blocks that leave sums of their own, from the sizes alone.
int64_t most_parts(int64_t rows, int64_t cols) {
    const int64_t n = cols <= 1024 ? 1216 : cols <= 2048 ? 608 : 304;
    return rows < n ? rows : n;
}

int64_t parts_of(int64_t rows) {  // of k_rms_columns
    const int64_t n = (rows + 63) / 64;
    return n < 64 ? n : 64;
}

template <typename T>
cudaError_t launch_typed(RmsBwd a, cudaStream_t stream) {
    a.parts = parts_of(a.rows);
    a.rows_per_part = (a.rows + a.parts - 1) / a.parts;
    const int64_t most = int64_t(1) << 30;
    cudaError_t e = launch_pdl(k_rms_dx<T>, dim3(unsigned(a.rows < most ? a.rows : most)), dim3(512), 0, stream, a);
    if (e != cudaSuccess) return e;
    const int64_t strips = (a.cols + 31) / 32;
    e = launch_pdl(k_rms_columns<T>, dim3(unsigned(strips < most ? strips : most), unsigned(a.parts)), dim3(256), 0, stream, a);
    if (e != cudaSuccess) return e;
    return launch_pdl(k_rms_join, dim3(unsigned(strips < (1 << 20) ? strips : (1 << 20))), dim3(256), 0, stream, a);
}

}  // namespace

// Debug builds: this unit's record of refused accesses.
TR_BOUNDS_READER(read_bounds_rmsnorm_backward)

cudaError_t launch_rmsnorm_backward(const tr_rmsnorm_backward_args &p) {
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(p.stream);
    if (p.rows == 0) return cudaMemsetAsync(p.dgamma, 0, size_t(p.cols) * 4, stream);  // the column sums are empty
    const RmsBwd a{p.dy, p.h, p.gamma, p.rstd, p.dresidual, p.dx, p.dgamma, static_cast<float *>(p.workspace),
                   p.rows, p.cols, p.ld_dy, p.ld_h, p.ld_dresidual, p.ld_dx, 0, 0, p.w_dtype == TR_DTYPE_BF16};
    return p.x_dtype == TR_DTYPE_F32 ? launch_typed<float>(a, stream) : launch_typed<__nv_bfloat16>(a, stream);
}

}  // namespace tr

extern "C" int64_t tr_rmsnorm_backward_workspace(int64_t rows, int64_t cols) {
    if (rows < 0 || cols < 0) return -1;
    if (rows == 0 || cols == 0) return 0;
    int64_t n;
    if (!tr::mul_add(cols, 4 * tr::most_parts(rows, cols), 0, &n)) return -1;
    return n;
}

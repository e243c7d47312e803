// Layer norm, backward: the input's gradient along the rows, the weight's and
// the bias's down the columns.
#include "launch.cuh"
#include "row_chunk.cuh"
#include "tr_internal.h"

namespace tr {
namespace {

struct Bwd {
    const void *dy, *x, *gamma;
    const float *mean, *rstd;
    void *dx;
    float *dgamma, *dbeta, *part;
    int64_t rows, cols, ld_dy, ld_x, ld_dx;
    int64_t parts, rows_per_part;
    bool w_bf16;
};

// dx of one row per block, in two walks along it.
template <typename T, int V>
__global__ void __launch_bounds__(512) k_ln_dx(Bwd a) {
    pdl_prologue();
    __shared__ float slots[2][64];
    int turn = 0;
    [[maybe_unused]] const dbg::Side sd = dbg::side(a.dy, 1, a.rows, a.cols, a.ld_dy, 0, sizeof(T));
    [[maybe_unused]] const dbg::Side sx = dbg::side(a.x, 1, a.rows, a.cols, a.ld_x, 0, sizeof(T));
    [[maybe_unused]] const dbg::Side so = dbg::side(a.dx, 1, a.rows, a.cols, a.ld_dx, 0, sizeof(T));
    [[maybe_unused]] const dbg::Side sw = dbg::side(a.gamma, 1, 1, a.cols, a.cols, 0, a.w_bf16 ? 2 : 4);
    [[maybe_unused]] const dbg::Side sm = dbg::side(a.mean, 1, 1, a.rows, a.rows, 0, 4);
    [[maybe_unused]] const dbg::Side sr = dbg::side(a.rstd, 1, 1, a.rows, a.rows, 0, 4);
    const float inv_cols = 1.0f / float(a.cols);
    const int64_t step = int64_t(blockDim.x) * V;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const T *dyr = static_cast<const T *>(a.dy) + row * a.ld_dy;
        const T *xr = static_cast<const T *>(a.x) + row * a.ld_x;
        T *dxr = static_cast<T *>(a.dx) + row * a.ld_dx;
        const float mean = TR_LOAD_OK(sm, a.mean + row, 4) ? a.mean[row] : 0.0f;
        const float rstd = TR_LOAD_OK(sr, a.rstd + row, 4) ? a.rstd[row] : 0.0f;
        const int64_t first = int64_t(threadIdx.x) * V - row_shift<T, V>(xr);
        float s1 = 0.0f, s2 = 0.0f;
        for (int64_t lo = first; lo < a.cols; lo += step) {
            const Pack<T, V> px = load_chunk<T, V>(xr, lo, a.cols, sx);
            const Pack<T, V> pd = load_chunk<T, V>(dyr, lo, a.cols, sd);
#pragma unroll
            for (int q = 0; q < V; ++q) {
                if (lo + q < 0 || lo + q >= a.cols) continue;
                const float g = pd.get(q) * weight(a.gamma, a.w_bf16, lo + q, sw);
                s1 += g;
                s2 = fmaf(g, (px.get(q) - mean) * rstd, s2);
            }
        }
        float s[2] = {s1, s2};
        group_sum<512, 2>(s, slots[turn]);
        turn ^= 1;
        s1 = s[0] * inv_cols;
        s2 = s[1] * inv_cols;
        for (int64_t lo = first; lo < a.cols; lo += step) {
            const Pack<T, V> px = load_chunk<T, V>(xr, lo, a.cols, sx);
            Pack<T, V> pd = load_chunk<T, V>(dyr, lo, a.cols, sd);
            float v[V];
#pragma unroll
            for (int q = 0; q < V; ++q) {
                v[q] = 0.0f;
                if (lo + q < 0 || lo + q >= a.cols) continue;
                const float g = pd.get(q) * weight(a.gamma, a.w_bf16, lo + q, sw);
                const float u = (px.get(q) - mean) * rstd;
                v[q] = rstd * (g - s1 - u * s2);
            }
            pd.round(v);
            store_chunk<T, V>(dxr, lo, a.cols, pd, so);
        }
    }
}

// Column sums of dy*u and dy over one part of the rows: 32 columns by 8 rows
// of threads, 2 x cols partial sums per part.
template <typename T>
__global__ void __launch_bounds__(256) k_ln_columns(Bwd a) {
    pdl_prologue();
    __shared__ float red[2][8][33];
    [[maybe_unused]] const dbg::Side sd = dbg::side(a.dy, 1, a.rows, a.cols, a.ld_dy, 0, sizeof(T));
    [[maybe_unused]] const dbg::Side sx = dbg::side(a.x, 1, a.rows, a.cols, a.ld_x, 0, sizeof(T));
    [[maybe_unused]] const dbg::Side sp = dbg::side(a.part, 1, 2 * a.parts, a.cols, a.cols, 0, 4);
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int64_t part = blockIdx.y;
    const int64_t r0 = part * a.rows_per_part;
    const int64_t r1 = r0 + a.rows_per_part < a.rows ? r0 + a.rows_per_part : a.rows;
    for (int64_t c0 = int64_t(blockIdx.x) * 32; c0 < a.cols; c0 += int64_t(gridDim.x) * 32) {
        const int64_t j = c0 + tx;
        float s1 = 0.0f, s2 = 0.0f;
        if (j < a.cols)
            for (int64_t r = r0 + ty; r < r1; r += 8) {
                const T *pd = static_cast<const T *>(a.dy) + r * a.ld_dy + j;
                const T *px = static_cast<const T *>(a.x) + r * a.ld_x + j;
                if (!TR_LOAD_OK(sd, pd, int(sizeof(T))) || !TR_LOAD_OK(sx, px, int(sizeof(T)))) continue;
                const float d = to_f32(*pd);
                s1 = fmaf(d, (to_f32(*px) - a.mean[r]) * a.rstd[r], s1);
                s2 += d;
            }
        red[0][ty][tx] = s1;
        red[1][ty][tx] = s2;
        __syncthreads();
        if (ty < 2 && j < a.cols) {
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) s += red[ty][i][tx];
            float *p = a.part + (part * 2 + ty) * a.cols + j;
            if (TR_STORE_OK(sp, p, 4)) *p = s;
        }
        __syncthreads();
    }
}

// The parts' sums, joined in their order.
__global__ void __launch_bounds__(256) k_ln_join(Bwd a) {
    pdl_prologue();
    [[maybe_unused]] const dbg::Side sp = dbg::side(a.part, 1, 2 * a.parts, a.cols, a.cols, 0, 4);
    [[maybe_unused]] const dbg::Side so = dbg::side(blockIdx.y ? a.dbeta : a.dgamma, 1, 1, a.cols, a.cols, 0, 4);
    float *out = blockIdx.y ? a.dbeta : a.dgamma;
    for (int64_t j = int64_t(blockIdx.x) * 256 + threadIdx.x; j < a.cols;
         j += int64_t(gridDim.x) * 256) {
        float s = 0.0f;
        for (int64_t i = 0; i < a.parts; ++i) {
            const float *p = a.part + (2 * i + blockIdx.y) * a.cols + j;
            if (TR_LOAD_OK(sp, p, 4)) s += *p;
        }
        if (TR_STORE_OK(so, out + j, 4)) out[j] = s;
    }
}

int64_t parts_of(int64_t rows) {
    const int64_t n = (rows + 63) / 64;
    return n < 64 ? n : 64;
}

template <typename T>
cudaError_t launch_typed(const Bwd &a, cudaStream_t stream) {
    constexpr int V = 16 / int(sizeof(T));
    const uintptr_t ax = reinterpret_cast<uintptr_t>(a.x), ad = reinterpret_cast<uintptr_t>(a.dy),
                    ao = reinterpret_cast<uintptr_t>(a.dx);
    const bool alike = (((ax ^ ad) | (ax ^ ao)) & 15u) == 0 &&
                       ((a.ld_x - a.ld_dy) * int64_t(sizeof(T))) % 16 == 0 &&
                       ((a.ld_x - a.ld_dx) * int64_t(sizeof(T))) % 16 == 0;
    const int64_t most = int64_t(1) << 30;
    const dim3 rows_grid(unsigned(a.rows < most ? a.rows : most));
    cudaError_t e = alike ? launch_pdl(k_ln_dx<T, V>, rows_grid, dim3(512), 0, stream, a)
                          : launch_pdl(k_ln_dx<T, 1>, rows_grid, dim3(512), 0, stream, a);
    if (e != cudaSuccess) return e;
    const int64_t strips = (a.cols + 31) / 32;
    const dim3 grid(unsigned(strips < most ? strips : most), unsigned(a.parts));
    return launch_pdl(k_ln_columns<T>, grid, dim3(256), 0, stream, a);
}

}  // namespace

// Debug builds: this unit's record of refused accesses.
TR_BOUNDS_READER(read_bounds_layernorm_backward)

cudaError_t launch_layernorm_backward(const tr_layernorm_backward_args &p) {
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(p.stream);
    if (p.rows == 0) {  // no rows: the column sums are empty
        cudaError_t e = cudaMemsetAsync(p.dgamma, 0, size_t(p.cols) * 4, stream);
        if (e == cudaSuccess && p.dbeta) e = cudaMemsetAsync(p.dbeta, 0, size_t(p.cols) * 4, stream);
        return e;
    }
    Bwd a{p.dy, p.x, p.gamma, p.mean, p.rstd, p.dx, p.dgamma, p.dbeta,
          static_cast<float *>(p.workspace), p.rows, p.cols, p.ld_dy, p.ld_x, p.ld_dx,
          parts_of(p.rows), 0, p.w_dtype == TR_DTYPE_BF16};
    a.rows_per_part = (p.rows + a.parts - 1) / a.parts;
    cudaError_t e = p.x_dtype == TR_DTYPE_F32 ? launch_typed<float>(a, stream)
                                              : launch_typed<__nv_bfloat16>(a, stream);
    if (e != cudaSuccess) return e;
    int64_t blocks = (p.cols + 255) / 256;
    if (blocks > 4096) blocks = 4096;
    return launch_pdl(k_ln_join, dim3(unsigned(blocks), p.dbeta ? 2 : 1), dim3(256), 0, stream, a);
}

}  // namespace tr

extern "C" int64_t tr_layernorm_backward_workspace(int64_t rows, int64_t cols) {
    if (rows < 0 || cols < 0) return -1;
    if (rows == 0 || cols == 0) return 0;
    int64_t n;
    if (!tr::mul_add(cols, 8 * tr::parts_of(rows), 0, &n)) return -1;
    return n;
}

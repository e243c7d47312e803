// Layer norm, forward: y = (x - mean) * rstd * gamma + beta along each row.
#include "launch.cuh"
#include "row_chunk.cuh"
#include "tr_internal.h"

namespace tr {
namespace {

struct Fwd {
    const void *x, *gamma, *beta;
    void *y;
    float *mean, *rstd;
    int64_t rows, cols, ld_x, ld_y;
    float eps, inv_cols;
    bool w_bf16;
};

// TPR threads hold R rows at a time, NCH chunks of each to a thread, in
// registers: x is read once, the deviations are summed about the mean from the
// registers, and a weight read serves R rows.  EDGE: rows or weights that do not
// start on 16-byte boundaries, or do not end on them.
template <typename T, int V, int TPR, int NCH, int R, bool EDGE>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR, EDGE || TPR > 512 ? 1 : 768 / (TPR < 128 ? 128 : TPR))
k_layernorm(const Fwd a) {
    pdl_prologue();
    constexpr int GROUPS = (TPR < 128 ? 128 : TPR) / TPR;
    __shared__ float slots[2][R * 32];
    const T *x = static_cast<const T *>(a.x);
    T *y = static_cast<T *>(a.y);
    [[maybe_unused]] const dbg::Side sx = dbg::side(x, 1, a.rows, a.cols, a.ld_x, 0, sizeof(T));
    [[maybe_unused]] const dbg::Side sy = dbg::side(y, 1, a.rows, a.cols, a.ld_y, 0, sizeof(T));
    [[maybe_unused]] const dbg::Side sw = dbg::side(a.gamma, 1, 1, a.cols, a.cols, 0, a.w_bf16 ? 2 : 4);
    [[maybe_unused]] const dbg::Side sb = dbg::side(a.beta, 1, 1, a.cols, a.cols, 0, a.w_bf16 ? 2 : 4);
    [[maybe_unused]] const dbg::Side ss = dbg::side(a.mean, 1, 1, a.rows, a.rows, 0, 4);
    [[maybe_unused]] const dbg::Side sr = dbg::side(a.rstd, 1, 1, a.rows, a.rows, 0, 4);
    const int t = threadIdx.x % TPR;
    const int cols = int(a.cols);  // a row that fits the registers
    for (int64_t row0 = (int64_t(blockIdx.x) * GROUPS + threadIdx.x / TPR) * R; row0 < a.rows;
         row0 += int64_t(gridDim.x) * GROUPS * R) {
        Pack<T, V> p[R][NCH];
        const int d = EDGE ? row_shift<T, V>(x + row0 * a.ld_x) : 0;
        static_assert(!EDGE || R == 1, "rows of their own shift go one at a time");
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const T *xr = x + (row0 + r) * a.ld_x;
#pragma unroll
            for (int i = 0; i < NCH; ++i)
                p[r][i] = load_chunk<T, V, EDGE>(xr, (t + i * TPR) * V - d, row0 + r < a.rows ? cols : 0, sx);
        }
        float mean[R], rstd[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            mean[r] = 0.0f;
#pragma unroll
            for (int i = 0; i < NCH; ++i)
#pragma unroll
                for (int q = 0; q < V; ++q) mean[r] += p[r][i].get(q);
        }
        group_sum<TPR, R>(mean, slots[0]);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            mean[r] *= a.inv_cols;
            rstd[r] = 0.0f;
#pragma unroll
            for (int i = 0; i < NCH; ++i) {
                const int lo = (t + i * TPR) * V - d;
                if (!EDGE && lo >= cols) continue;
                p[r][i].forget();
#pragma unroll
                for (int q = 0; q < V; ++q) {
                    const float o = p[r][i].get(q) - mean[r];
                    if (!EDGE || (lo + q >= 0 && lo + q < cols)) rstd[r] = fmaf(o, o, rstd[r]);
                }
            }
        }
        group_sum<TPR, R>(rstd, slots[1]);
#pragma unroll
        for (int r = 0; r < R; ++r) rstd[r] = 1.0f / sqrtf(fmaf(rstd[r], a.inv_cols, a.eps));
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const int lo = (t + i * TPR) * V - d;
            if (lo >= cols) continue;
            float w[V], b[V];
            if constexpr (EDGE) {
#pragma unroll
                for (int q = 0; q < V; ++q) {
                    const bool in = lo + q >= 0 && lo + q < cols;
                    w[q] = in ? weight(a.gamma, a.w_bf16, lo + q, sw) : 0.0f;
                    b[q] = in && a.beta ? weight(a.beta, a.w_bf16, lo + q, sb) : 0.0f;
                }
            } else {
                load_weights<V>(a.gamma, a.w_bf16, lo, w, sw);
                if (a.beta) load_weights<V>(a.beta, a.w_bf16, lo, b, sb);
            }
#pragma unroll
            for (int r = 0; r < R; ++r) {
                if (row0 + r >= a.rows) continue;
                Pack<T, V> o;
                float v[V];
                p[r][i].forget();
#pragma unroll
                for (int q = 0; q < V; ++q) {
                    const float u = (p[r][i].get(q) - mean[r]) * rstd[r];
                    v[q] = a.beta ? fmaf(u, w[q], b[q]) : u * w[q];
                }
                o.round(v);
                store_chunk<T, V, EDGE>(y + (row0 + r) * a.ld_y, lo, cols, o, sy);
            }
        }
        if (t == 0)
#pragma unroll
            for (int r = 0; r < R; ++r) {
                if (row0 + r >= a.rows) continue;
                if (a.mean && TR_STORE_OK(ss, a.mean + row0 + r, 4)) a.mean[row0 + r] = mean[r];
                if (a.rstd && TR_STORE_OK(sr, a.rstd + row0 + r, 4)) a.rstd[row0 + r] = rstd[r];
            }
    }
}

// Rows too long for registers, and rows whose x and y are offset differently
// from a 16-byte boundary (V = 1): a block walks its row three times.
template <typename T, int V>
__global__ void __launch_bounds__(1024) k_layernorm_long(const Fwd a) {
    pdl_prologue();
    __shared__ float slots[2][32];
    const T *x = static_cast<const T *>(a.x);
    T *y = static_cast<T *>(a.y);
    const int64_t cols = a.cols;
    [[maybe_unused]] const dbg::Side sx = dbg::side(x, 1, a.rows, cols, a.ld_x, 0, sizeof(T));
    [[maybe_unused]] const dbg::Side sy = dbg::side(y, 1, a.rows, cols, a.ld_y, 0, sizeof(T));
    [[maybe_unused]] const dbg::Side sw = dbg::side(a.gamma, 1, 1, cols, cols, 0, a.w_bf16 ? 2 : 4);
    [[maybe_unused]] const dbg::Side sb = dbg::side(a.beta, 1, 1, cols, cols, 0, a.w_bf16 ? 2 : 4);
    [[maybe_unused]] const dbg::Side ss = dbg::side(a.mean, 1, 1, a.rows, a.rows, 0, 4);
    [[maybe_unused]] const dbg::Side sr = dbg::side(a.rstd, 1, 1, a.rows, a.rows, 0, 4);
    const int64_t step = int64_t(blockDim.x) * V;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const T *xr = x + row * a.ld_x;
        const int64_t first = int64_t(threadIdx.x) * V - row_shift<T, V>(xr);
        float mean[1] = {0.0f}, rstd[1] = {0.0f};
        for (int64_t lo = first; lo < cols; lo += step) {
            const Pack<T, V> p = load_chunk<T, V>(xr, lo, cols, sx);
#pragma unroll
            for (int q = 0; q < V; ++q) mean[0] += p.get(q);
        }
        group_sum<1024, 1>(mean, slots[0]);
        mean[0] *= a.inv_cols;
        for (int64_t lo = first; lo < cols; lo += step) {
            const Pack<T, V> p = load_chunk<T, V>(xr, lo, cols, sx);
#pragma unroll
            for (int q = 0; q < V; ++q) {
                const float o = p.get(q) - mean[0];
                if (lo + q >= 0 && lo + q < cols) rstd[0] = fmaf(o, o, rstd[0]);
            }
        }
        group_sum<1024, 1>(rstd, slots[1]);
        rstd[0] = 1.0f / sqrtf(fmaf(rstd[0], a.inv_cols, a.eps));
        T *yr = y + row * a.ld_y;
        for (int64_t lo = first; lo < cols; lo += step) {
            Pack<T, V> p = load_chunk<T, V>(xr, lo, cols, sx);
            float v[V];
#pragma unroll
            for (int q = 0; q < V; ++q) {
                const int64_t j = lo + q;
                v[q] = 0.0f;
                if (j < 0 || j >= cols) continue;
                v[q] = (p.get(q) - mean[0]) * rstd[0] * weight(a.gamma, a.w_bf16, j, sw);
                if (a.beta) v[q] += weight(a.beta, a.w_bf16, j, sb);
            }
            p.round(v);
            store_chunk<T, V>(yr, lo, cols, p, sy);
        }
        if (threadIdx.x == 0) {
            if (a.mean && TR_STORE_OK(ss, a.mean + row, 4)) a.mean[row] = mean[0];
            if (a.rstd && TR_STORE_OK(sr, a.rstd + row, 4)) a.rstd[row] = rstd[0];
        }
    }
}

template <typename T>
cudaError_t launch_typed(const tr_layernorm_args &p) {
    constexpr int V = 16 / int(sizeof(T));
    constexpr int es = int(sizeof(T));
    const uintptr_t ax = reinterpret_cast<uintptr_t>(p.x), ay = reinterpret_cast<uintptr_t>(p.y);
    const bool alike = ((ax ^ ay) & 15u) == 0 && ((p.ld_x - p.ld_y) * es) % 16 == 0;
    const bool shifted = (ax & 15u) != 0 || (p.ld_x * es) % 16 != 0;
    const uintptr_t aw = reinterpret_cast<uintptr_t>(p.gamma) | reinterpret_cast<uintptr_t>(p.beta);
    const Fwd a{p.x, p.gamma, p.beta, p.y, p.mean, p.rstd, p.rows, p.cols, p.ld_x, p.ld_y, p.eps,
                1.0f / float(p.cols), p.w_dtype == TR_DTYPE_BF16};
    const bool edge = shifted || p.cols % V != 0 || (aw & 15u) != 0;
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(p.stream);
    auto run = [&](auto kern, int threads, int rows_per_block) {
        const int64_t most = int64_t(1) << 30;
        int64_t grid = (a.rows + rows_per_block - 1) / rows_per_block;
        if (grid > most) grid = most;
        return launch_pdl(kern, dim3(unsigned(grid)), dim3(threads), 0, stream, a);
    };
    if (!alike) return run(k_layernorm_long<T, 1>, 1024, 1);
    const int64_t chunks = (a.cols + (shifted ? V - 1 : 0) + V - 1) / V;
    const bool many = a.rows >= int64_t(sm_count()) * 16;  // two rows to a block still fill the machine
#define TR_ROWS(TPR, NCH, BLOCK)                                                              \
    if (chunks <= TPR * NCH)                                                                  \
        return edge   ? run(k_layernorm<T, V, TPR, NCH, 1, true>, BLOCK, BLOCK / TPR)         \
               : many ? run(k_layernorm<T, V, TPR, NCH, 2, false>, BLOCK, 2 * BLOCK / TPR)    \
                      : run(k_layernorm<T, V, TPR, NCH, 1, false>, BLOCK, BLOCK / TPR);
    TR_ROWS(32, 1, 128)
    TR_ROWS(32, 2, 128)
    TR_ROWS(32, 4, 128)
    TR_ROWS(128, 2, 128)
    TR_ROWS(128, 4, 128)
    TR_ROWS(256, 4, 256)
    TR_ROWS(512, 4, 512)
#undef TR_ROWS
    if (chunks <= 4096)
        return edge ? run(k_layernorm<T, V, 1024, 4, 1, true>, 1024, 1) : run(k_layernorm<T, V, 1024, 4, 1, false>, 1024, 1);
    return run(k_layernorm_long<T, V>, 1024, 1);
}

}  // namespace

// Debug builds: this unit's record of refused accesses.
TR_BOUNDS_READER(read_bounds_layernorm)

cudaError_t launch_layernorm(const tr_layernorm_args &a) {
    return a.x_dtype == TR_DTYPE_F32 ? launch_typed<float>(a) : launch_typed<__nv_bfloat16>(a);
}

}  // namespace tr

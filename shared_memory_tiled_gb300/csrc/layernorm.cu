// Layer norm, forward: y = (x - mean) * rstd * gamma + beta along each row, with
// mean = sum(x) / n and rstd = 1 / sqrt(sum((x - mean)^2) / n + eps).
//
// Bound by memory: one read of x and one write of y.  Every kernel but the last
// resort therefore holds a row in registers between its three walks (sum,
// deviations about the mean, output).  Summing the squares with the values would
// save a walk and lose the variance of a row with a large mean.
//
// Measured on one GB300 (share of the measured copy rate, 6771 GB/s):
//   16384 x 8192 bf16, fp32 weights   88 us, 6.1 TB/s (91%)
//   16384 x 8192 fp32                181 us, 5.9 TB/s (88%)
//   65536 x 1024 bf16                 45 us, 5.9 TB/s (88%)
//   12289 x 7919 fp32 (rows off 16-byte boundaries)  155 us, 5.0 TB/s (74%)
//   1 x 8192 bf16                    4.1 us: a launch and three trips to memory
//   1024, 2048, 4096 x 8192 bf16     11.6, 17.7, 32.0 us: 2.9, 3.8, 4.2 TB/s (weights from L1)
//   4096 x 32768 bf16 / fp32         168 / 278 us, 3.2 / 3.9 TB/s (the row is walked three times)
//   8192 x 5003 bf16, x padded and y not  192 us, 0.9 TB/s (one value to an access)
#include "launch.cuh"
#include "row_chunk.cuh"
#include "tr_internal.h"
namespace tr {
namespace {

constexpr int kMostRowChunks = 2049;  // of a row whose weights are kept in shared memory, one for the shift

struct Fwd {
    const void *x, *gamma, *beta;
    void *y;
    float *mean, *rstd;
    int64_t rows, cols, ld_x, ld_y;
    float eps, inv_cols;
    bool w_bf16;
};

// Few rows: TPR threads hold one row, NCH chunks to a thread, in registers, so that
// x is read once; the deviations are summed about the mean from the registers.
// EDGE: rows or weights that do not start on 16-byte boundaries, or do not end on
// them.
template <typename T, int V, int TPR, int NCH, bool EDGE>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR) k_layernorm(const Fwd a) {
    pdl_prologue();
    constexpr int GROUPS = (TPR < 128 ? 128 : TPR) / TPR;
    __shared__ float slots[2][32];
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
    const uint32_t z1 = opaque_zero_1(), z2 = opaque_zero_2();
    for (int64_t row = int64_t(blockIdx.x) * GROUPS + threadIdx.x / TPR; row < a.rows;
         row += int64_t(gridDim.x) * GROUPS) {
        const T *xr = x + row * a.ld_x;
        const int d = EDGE ? row_shift<T, V>(xr) : 0;
        Pack<T, V> p[NCH];
#pragma unroll
        for (int i = 0; i < NCH; ++i) p[i] = load_chunk<T, V, EDGE>(xr, (t + i * TPR) * V - d, cols, sx);
        float mean[1] = {0.0f}, rstd[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < NCH; ++i)
#pragma unroll
            for (int q = 0; q < V; ++q) mean[0] += p[i].get(q);
        group_sum<TPR, 1>(mean, slots[0]);
        mean[0] *= a.inv_cols;
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const int lo = (t + i * TPR) * V - d;
            if (!EDGE && lo >= cols) continue;
#pragma unroll
            for (int q = 0; q < V; ++q) {
                const float o = p[i].get(q, z1) - mean[0];
                if (!EDGE || (lo + q >= 0 && lo + q < cols)) rstd[0] = fmaf(o, o, rstd[0]);
            }
        }
        group_sum<TPR, 1>(rstd, slots[1]);
        rstd[0] = 1.0f / sqrtf(fmaf(rstd[0], a.inv_cols, a.eps));
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const int lo = (t + i * TPR) * V - d;
            if (lo >= cols) continue;
            float w[V], b[V], v[V];
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
            Pack<T, V> o;
#pragma unroll
            for (int q = 0; q < V; ++q) {
                const float u = (p[i].get(q, z2) - mean[0]) * rstd[0];
                v[q] = a.beta ? fmaf(u, w[q], b[q]) : u * w[q];
            }
            o.round(v);
            store_chunk<T, V, EDGE>(y + row * a.ld_y, lo, cols, o, sy);
        }
        if (t == 0) {
            if (a.mean && TR_STORE_OK(ss, a.mean + row, 4)) a.mean[row] = mean[0];
            if (a.rstd && TR_STORE_OK(sr, a.rstd + row, 4)) a.rstd[row] = rstd[0];
        }
    }
}

// Many rows: a resident block walks the rows, G threads (one warp, or a few with
// a named barrier of their own) to a row, so that a row's loads, sums and stores
// run beside those of the block's other rows and no barrier stops them all.  The
// weights are read from memory once per block and kept in shared memory in
// fp32, laid out so that a warp's reads share no bank: without EDGE the V weights
// of a chunk in groups of 4, group h of chunk c at 4 * (h * chunks + c); with EDGE
// weight j at (j % V) * chunks + j / V, which any shift of the row leaves in
// neighbouring words.
//
// Why: with a block to each row and the weights read from L1 (8 fp32 bytes for every
// 4 bytes of x and y) 16384 x 8192 bf16 took 121 us.  The shape for 8192 bf16 is
// 4 warps to a row, 8 chunks to a thread, 6 rows to a block (88 us): 1 warp to a row
// takes 113 us (its 32 chunks leave room for 12 rows' loads only), 2 warps 101, 8
// warps 93, 4 warps and 8 rows 91.
template <typename T, int V, int G, int NCH, bool EDGE>
__global__ void __launch_bounds__(G == 32 && NCH <= 8 ? 1024 : NCH <= 8 ? 768 : 640, 1) k_layernorm_rows(const Fwd a) {
    extern __shared__ float4 weights4[];
    __shared__ float slots[2][32];
    float *gamma = reinterpret_cast<float *>(weights4);
    const int cols = int(a.cols);
    const int chunks = (cols + V - 1) / V + (EDGE ? 1 : 0);
    float *beta = gamma + chunks * V;
    const T *x = static_cast<const T *>(a.x);
    T *y = static_cast<T *>(a.y);
    [[maybe_unused]] const dbg::Side sx = dbg::side(x, 1, a.rows, a.cols, a.ld_x, 0, sizeof(T));
    [[maybe_unused]] const dbg::Side sy = dbg::side(y, 1, a.rows, a.cols, a.ld_y, 0, sizeof(T));
    [[maybe_unused]] const dbg::Side sw = dbg::side(a.gamma, 1, 1, a.cols, a.cols, 0, a.w_bf16 ? 2 : 4);
    [[maybe_unused]] const dbg::Side sb = dbg::side(a.beta, 1, 1, a.cols, a.cols, 0, a.w_bf16 ? 2 : 4);
    [[maybe_unused]] const dbg::Side ss = dbg::side(a.mean, 1, 1, a.rows, a.rows, 0, 4);
    [[maybe_unused]] const dbg::Side sr = dbg::side(a.rstd, 1, 1, a.rows, a.rows, 0, 4);
    pdl_prologue();
    auto place = [&](int j) {
        return EDGE ? j % V * chunks + j / V : 4 * (j % V / 4 * chunks + j / V) + j % 4;
    };
    for (int j = threadIdx.x; j < cols; j += blockDim.x) {
        gamma[place(j)] = weight(a.gamma, a.w_bf16, j, sw);
        if (a.beta) beta[place(j)] = weight(a.beta, a.w_bf16, j, sb);
    }
    __syncthreads();
    const int group = threadIdx.x / G, groups = blockDim.x / G, t = threadIdx.x % G;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t z1 = opaque_zero_1(), z2 = opaque_zero_2();
    auto sum = [&](float v, int slot) {
        v = warp_sum(v);
        if constexpr (G > 32) {
            if (lane == 0) slots[slot][warp] = v;
            asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(G) : "memory");
            v = slots[slot][group * (G / 32)];
#pragma unroll
            for (int k = 1; k < G / 32; ++k) v += slots[slot][group * (G / 32) + k];
        }
        return v;
    };
    for (int64_t row = int64_t(blockIdx.x) * groups + group; row < a.rows; row += int64_t(gridDim.x) * groups) {
        const T *xr = x + row * a.ld_x;
        const int d = EDGE ? row_shift<T, V>(xr) : 0;
        Pack<T, V> p[NCH];
#pragma unroll
        for (int i = 0; i < NCH; ++i) p[i] = load_chunk<T, V, EDGE>(xr, (t + i * G) * V - d, cols, sx);
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            float part = 0.0f;
#pragma unroll
            for (int q = 0; q < V; ++q) part += p[i].get(q);
            s += part;
        }
        const float mean = sum(s, 0) * a.inv_cols;
        s = 0.0f;
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const int lo = (t + i * G) * V - d;
            if (!EDGE && lo >= cols) continue;
            float part = 0.0f;
#pragma unroll
            for (int q = 0; q < V; ++q) {
                const float o = p[i].get(q, z1) - mean;
                if (!EDGE || (lo + q >= 0 && lo + q < cols)) part = fmaf(o, o, part);
            }
            s += part;
        }
        const float rstd = 1.0f / sqrtf(fmaf(sum(s, 1), a.inv_cols, a.eps));
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const int c = t + i * G, lo = c * V - d;
            if (lo >= cols) continue;
            float v[V];
#pragma unroll
            for (int q = 0; q < V; ++q) v[q] = (p[i].get(q, z2) - mean) * rstd;
            if constexpr (EDGE) {
#pragma unroll
                for (int q = 0; q < V; ++q) {
                    if (lo + q < 0 || lo + q >= cols) continue;
                    const int at = place(lo + q);
                    v[q] = a.beta ? fmaf(v[q], gamma[at], beta[at]) : v[q] * gamma[at];
                }
            } else {
#pragma unroll
                for (int h = 0; h < V / 4; ++h) {
                    const float4 w = weights4[h * chunks + c];
                    const float4 b = a.beta ? weights4[chunks * (V / 4) + h * chunks + c] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    v[4 * h] = fmaf(v[4 * h], w.x, b.x);
                    v[4 * h + 1] = fmaf(v[4 * h + 1], w.y, b.y);
                    v[4 * h + 2] = fmaf(v[4 * h + 2], w.z, b.z);
                    v[4 * h + 3] = fmaf(v[4 * h + 3], w.w, b.w);
                }
            }
            Pack<T, V> o;
            o.round(v);
            store_chunk<T, V, EDGE>(y + row * a.ld_y, lo, cols, o, sy);
        }
        if (t == 0) {
            if (a.mean && TR_STORE_OK(ss, a.mean + row, 4)) a.mean[row] = mean;
            if (a.rstd && TR_STORE_OK(sr, a.rstd + row, 4)) a.rstd[row] = rstd;
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

// One block to an SM, with its copy of the weights.
template <typename K>
cudaError_t launch_rows(K kern, int threads, int v, const Fwd &a, bool edge, cudaStream_t stream) {
    const int64_t chunks = (a.cols + v - 1) / v + (edge ? 1 : 0);
    const size_t smem = size_t(chunks) * v * 4 * (a.beta ? 2 : 1);
    // Always the most that any call needs: threads with rows of other lengths set it too.
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostRowChunks * 8 * 4 * 2);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3(unsigned(sm_count())), dim3(threads), smem, stream, a);
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
    // Rows for every group of every resident block, counted in the shape with most groups:
    // the weights' copy pays (8192 bf16: 4864 rows 32.1 us with it, 4863 rows 38.2 without;
    // where it begins to pay for the other shapes was not measured).
    if (a.rows >= int64_t(sm_count()) * 32 && chunks < kMostRowChunks) {
#define TR_ROWS(G, NCH, BLOCK)                                                            \
    if (chunks <= G * NCH)                                                                \
        return edge ? launch_rows(k_layernorm_rows<T, V, G, NCH, true>, BLOCK, V, a, true, stream) \
                    : launch_rows(k_layernorm_rows<T, V, G, NCH, false>, BLOCK, V, a, false, stream);
        TR_ROWS(32, 4, 1024)
        TR_ROWS(32, 8, 1024)
        TR_ROWS(32, 16, 640)
        TR_ROWS(128, 8, 768)
        TR_ROWS(128, 16, 640)
#undef TR_ROWS
    }
#define TR_ROWS(TPR, NCH, BLOCK)                                                              \
    if (chunks <= TPR * NCH)                                                                  \
        return edge ? run(k_layernorm<T, V, TPR, NCH, true>, BLOCK, BLOCK / TPR)              \
                    : run(k_layernorm<T, V, TPR, NCH, false>, BLOCK, BLOCK / TPR);
    TR_ROWS(32, 1, 128)
    TR_ROWS(32, 4, 128)
    TR_ROWS(128, 4, 128)
    TR_ROWS(256, 4, 256)
    TR_ROWS(512, 4, 512)
    TR_ROWS(1024, 4, 1024)
#undef TR_ROWS
    return run(k_layernorm_long<T, V>, 1024, 1);
}

}  // namespace

// Debug builds: this unit's record of refused accesses.
TR_BOUNDS_READER(read_bounds_layernorm)

cudaError_t launch_layernorm(const tr_layernorm_args &a) {
    return a.x_dtype == TR_DTYPE_F32 ? launch_typed<float>(a) : launch_typed<__nv_bfloat16>(a);
}

}  // namespace tr

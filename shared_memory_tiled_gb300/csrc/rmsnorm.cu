// Root-mean-square norm with the residual's addition: h = x + residual, and
// y = h * rstd * gamma with rstd = 1 / sqrt(sum(h^2) / n + eps), as rows of h's type and in
// 8 bits with a scale for each block of 128, by rows and transposed.
//
// Bound by memory: x and residual are read once, h, y, q and qt written once.
#include <type_traits>

#include "fp8.cuh"
#include "launch.cuh"
#include "ptx.cuh"
#include "row_chunk.cuh"
#include "row_ring.cuh"
#include "tr_internal.h"
#include "wait_selftest.cuh"

namespace tr {

// Set when a bounded in-kernel wait ran out; read and cleared by the host.
__device__ unsigned g_fault_flag_rmsnorm = 0;

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

// What a kernel stores its rows through.
struct RmsSides {
    dbg::Side x, res, h, y, w, rstd, q, scale;
};
template <typename T>
__device__ __forceinline__ RmsSides sides_of(const Rms &a) {
    return RmsSides{dbg::side(a.x, 1, a.rows, a.cols, a.ld_x, 0, sizeof(T)),
                    dbg::side(a.residual, 1, a.rows, a.cols, a.ld_residual, 0, sizeof(T)),
                    dbg::side(a.h, 1, a.rows, a.cols, a.ld_h, 0, sizeof(T)),
                    dbg::side(a.y, 1, a.rows, a.cols, a.ld_y, 0, sizeof(T)),
                    dbg::side(a.gamma, 1, 1, a.cols, a.cols, 0, a.w_bf16 ? 2 : 4),
                    dbg::side(a.rstd, 1, 1, a.rows, a.rows, 0, 4),
                    dbg::side(a.q, 1, a.rows, a.cols, a.ld_q, 0, 1),
                    dbg::side(a.scale, 1, (a.cols + 127) / 128, a.rows, a.ld_scale, 0, 4)};
}

__device__ __forceinline__ uint32_t bits_of(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// The larger of a and |b|; a NaN wins.
__device__ __forceinline__ float max_abs(float a, float b) {
    float m;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(fabsf(b)));
    return m;
}
constexpr float kFloor = 0x1p-100f;  // kFloorBits

// y = h * rstd * w for N values, two to an instruction.
template <int N>
__device__ __forceinline__ void normed(float (&y)[N], const float (&h)[N], float rstd, const float (&w)[N]) {
#pragma unroll
    for (int q = 0; q < N; q += 2) {
        const float2 v = __fmul2_rn(__fmul2_rn(make_float2(h[q], h[q + 1]), make_float2(rstd, rstd)), make_float2(w[q], w[q + 1]));
        y[q] = v.x;
        y[q + 1] = v.y;
    }
}

// V values times r as V bytes in words.
template <bool E5M2, int V>
__device__ __forceinline__ void to_words(uint32_t (&w)[V / 4], const float (&y)[V], float r) {
    constexpr __nv_fp8_interpretation_t K = E5M2 ? __NV_E5M2 : __NV_E4M3;
#pragma unroll
    for (int k = 0; k < V / 4; ++k) {
        const float2 a = __fmul2_rn(make_float2(y[4 * k], y[4 * k + 1]), make_float2(r, r));
        const float2 b = __fmul2_rn(make_float2(y[4 * k + 2], y[4 * k + 3]), make_float2(r, r));
        w[k] = uint32_t(__nv_cvt_float2_to_fp8x2(a, __NV_SATFINITE, K)) | uint32_t(__nv_cvt_float2_to_fp8x2(b, __NV_SATFINITE, K)) << 16;
    }
}

// Quantizes N chunks of V values of row `row`, the chunk n from column lo[n] (a multiple of V) on, each one's block of
// 128 held by the 128 / V neighbouring lanes; those past the row's end are zero and not stored.  A warp has N * V / 4
// blocks: as many lanes find one's T / a and as many its a / T, with one division's instructions for all of them
// (a division in each lane for each chunk: 163 us against 150 for 16384 x 8192 bf16, rows alone).
template <int V, int N>
__device__ __forceinline__ void quantize_chunks(const Rms &a, int64_t row, const int (&lo)[N], const float (&y)[N][V], const RmsSides &s) {
    constexpr int LANES = 128 / V, BLOCKS = 32 / LANES;  // blocks of a warp to a chunk
    const int lane = threadIdx.x & 31;
    float m[N], mine = kFloor;
#pragma unroll
    for (int n = 0; n < N; ++n) {
        m[n] = kFloor;
#pragma unroll
        for (int q = 0; q < V; ++q) m[n] = max_abs(m[n], y[n][q]);
#pragma unroll
        for (int o = LANES / 2; o; o >>= 1) m[n] = max_abs(m[n], __shfl_xor_sync(0xffffffffu, m[n], o));
        // Block b of chunk n goes to lane n * BLOCKS + b, and to the one 16 further.
        const float f = BLOCKS == 1 ? m[n] : __shfl_sync(0xffffffffu, m[n], (lane & (BLOCKS - 1)) * LANES);
        if ((lane & 15) / BLOCKS == n) mine = f;
    }
    const bool inverse = lane < 16;
    const float ratio = (inverse ? a.top : mine) / (inverse ? mine : a.top);
    // a / T: lane 16 + n * BLOCKS + b stores block b of chunk n.
    {
        const int n = (lane & 15) / BLOCKS, b = lane & (BLOCKS - 1);
        int col = 0;
#pragma unroll
        for (int k = 0; k < N; ++k)
            if (k == n) col = lo[k] - lane * V + b * 128;  // the warp's first column of that chunk, and the block's
        if (!inverse && n < N && col < a.cols) {
            float *p = a.scale + int64_t(col >> 7) * a.ld_scale + row;
            if (TR_STORE_OK(s.scale, p, 4)) *p = ratio;
        }
    }
    uint8_t *out = a.q + row * a.ld_q;
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const float inv = __shfl_sync(0xffffffffu, ratio, n * BLOCKS + lane / LANES);
        uint32_t w[V / 4];
        if (a.e5m2) to_words<true, V>(w, y[n], inv);
        else to_words<false, V>(w, y[n], inv);
        if (lo[n] >= a.cols) continue;
        if constexpr (V == 8) {
            if (TR_STORE_OK(s.q, out + lo[n], 8)) *reinterpret_cast<uint2 *>(out + lo[n]) = make_uint2(w[0], w[1]);
        } else {
            if (TR_STORE_OK(s.q, out + lo[n], 4)) *reinterpret_cast<uint32_t *>(out + lo[n]) = w[0];
        }
    }
}

// Sum over the block, in every thread; `slot` holds a word for each of 32 warps.
__device__ __forceinline__ float block_sum(float v, float *slot) {
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    v = warp_sum(v);
    if (lane == 0) slot[threadIdx.x >> 5] = v;
    __syncthreads();
    return warp_sum(lane < warps ? slot[lane] : 0.0f);
}

// Short rows, and few rows of up to 2048 chunks: TPR threads hold one row, NCH chunks of 16 bytes to a thread, and
// its weights, in registers.  Rows, weights and their ends on 16-byte boundaries.
template <typename T, int TPR, int NCH>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR) k_rmsnorm_held(const Rms a) {
    pdl_prologue();
    constexpr int V = 16 / int(sizeof(T)), GROUPS = (TPR < 128 ? 128 : TPR) / TPR;
    __shared__ float slots[2][32];
    const RmsSides s = sides_of<T>(a);
    const int t = threadIdx.x % TPR, cols = int(a.cols);
    float w[NCH][V];
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
        const int lo = (t + i * TPR) * V;
#pragma unroll
        for (int q = 0; q < V; ++q) w[i][q] = 0.0f;
        if (lo < cols) load_weights<V>(a.gamma, a.w_bf16, lo, w[i], s.w);
    }
    int turn = 0;
    for (int64_t row = int64_t(blockIdx.x) * GROUPS + threadIdx.x / TPR; row < a.rows; row += int64_t(gridDim.x) * GROUPS, turn ^= 1) {
        Pack<T, V> h[NCH], r[NCH];
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const int lo = (t + i * TPR) * V;
            h[i] = load_chunk<T, V, false>(static_cast<const T *>(a.x) + row * a.ld_x, lo, cols, s.x);
            if (a.residual) r[i] = load_chunk<T, V, false>(static_cast<const T *>(a.residual) + row * a.ld_residual, lo, cols, s.res);
        }
        float sum[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const int lo = (t + i * TPR) * V;
            if (a.residual) {
                float v[V];
#pragma unroll
                for (int q = 0; q < V; ++q) v[q] = h[i].get(q) + r[i].get(q);
                h[i].round(v);
                if (lo < cols) store_chunk<T, V, false>(static_cast<T *>(a.h) + row * a.ld_h, lo, cols, h[i], s.h);
            }
#pragma unroll
            for (int q = 0; q < V; ++q) sum[0] = fmaf(h[i].get(q), h[i].get(q), sum[0]);
        }
        group_sum<TPR, 1>(sum, slots[turn]);
        const float rstd = 1.0f / sqrtf(fmaf(sum[0], a.inv_cols, a.eps));
        if (t == 0 && a.rstd && TR_STORE_OK(s.rstd, a.rstd + row, 4)) a.rstd[row] = rstd;
        float y[NCH][V];
        int lo[NCH];
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            lo[i] = (t + i * TPR) * V;
            float v[V];
#pragma unroll
            for (int q = 0; q < V; ++q) v[q] = h[i].get(q);
            normed<V>(y[i], v, rstd, w[i]);
            if (a.y && lo[i] < cols) {
                Pack<T, V> o;
                o.round(y[i]);
                store_chunk<T, V, false>(static_cast<T *>(a.y) + row * a.ld_y, lo[i], cols, o, s.y);
            }
        }
        if (a.q) quantize_chunks<V, NCH>(a, row, lo, y, s);
    }
}

// Many rows: a block walks every n-th row; bulk copies keep a ring of its next rows of x and residual in flight,
// so no register holds loaded data and any alignment reads whole granules.  A thread owns the same 16
// columns of every row, their weights in registers.  VEC: columns in 16-byte chunks, every row on a
// 16-byte boundary; else a warp owns blocks of 128 columns and a lane every 32nd of them.
template <typename T, bool VEC>
__global__ void __launch_bounds__(1024, 1) k_rmsnorm_ring(const Rms a, int stages, uint32_t row_bytes) {
    constexpr int V = VEC ? 16 / int(sizeof(T)) : 4;  // columns that are quantized together
    constexpr int N = 16 / V;
    extern __shared__ uint4 ring4[];
    __shared__ uint64_t full[kMaxStages];
    __shared__ float slots[2][32];
    uint8_t *ring = reinterpret_cast<uint8_t *>(ring4);
    const RmsSides s = sides_of<T>(a);
    const int t = threadIdx.x, nt = blockDim.x, lane = t & 31, cols = int(a.cols);
    const bool add = a.residual != nullptr;
    const uint32_t stage_bytes = add ? 2 * row_bytes : row_bytes;
    if (t == 0) {
        for (int i = 0; i < stages; ++i) ptx::mbar_init(full + i, 1);
        ptx::fence_barrier_init();
    }
    __syncthreads();
    pdl_prologue();
    auto issue = [&](int64_t row, int stage) {  // one thread
        const Granules gx = granules<T>(a.x, a.rows, a.cols, a.ld_x, row);
        const Granules gr = add ? granules<T>(a.residual, a.rows, a.cols, a.ld_residual, row) : Granules{nullptr, 0, 0, true};
        uint8_t *at = ring + size_t(stage) * stage_bytes;
        if (!gx.inside || !gr.inside) {  // the block copies that row itself
            ptx::mbar_arrive(full + stage);
            return;
        }
        ptx::mbar_arrive_expect_tx(full + stage, gx.bytes + gr.bytes);
        ptx::bulk_load(at, gx.src, gx.bytes, full + stage);
        if (add) ptx::bulk_load(at + row_bytes, gr.src, gr.bytes, full + stage);
    };
    if (t == 0)
        for (int i = 0; i < stages && blockIdx.x + int64_t(i) * gridDim.x < a.rows; ++i)
            issue(blockIdx.x + int64_t(i) * gridDim.x, i);
    // Column of value q of the thread's piece i.
    auto column = [&](int i, int q) {
        return VEC ? (t + i * nt) * V + q : (i * (nt >> 5) + (t >> 5)) * 128 + q * 32 + lane;
    };
    float w[N][V];
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int q = 0; q < V; ++q) {
            const int j = column(i, q);
            w[i][q] = j < cols ? weight(a.gamma, a.w_bf16, j, s.w) : 0.0f;
        }
    bool ok = true;
    int stage = 0, turn = 0;
    uint32_t phase = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        if (ok) ok = ptx::mbar_wait_bounded(full + stage, phase);
        uint8_t *at = ring + size_t(stage) * stage_bytes;
        T *px = reinterpret_cast<T *>(at), *pr = reinterpret_cast<T *>(at + row_bytes);
        if constexpr (!VEC) {
            const Granules gx = granules<T>(a.x, a.rows, a.cols, a.ld_x, row);
            const Granules gr = add ? granules<T>(a.residual, a.rows, a.cols, a.ld_residual, row) : Granules{nullptr, 0, 0, true};
            px = reinterpret_cast<T *>(at + gx.shift);
            pr = reinterpret_cast<T *>(at + row_bytes + gr.shift);
            if (!gx.inside || !gr.inside) {
                const T *xr = static_cast<const T *>(a.x) + row * a.ld_x;
                const T *rr = static_cast<const T *>(a.residual) + row * a.ld_residual;
                for (int j = t; j < cols; j += nt) {
                    if (TR_LOAD_OK(s.x, xr + j, int(sizeof(T)))) px[j] = xr[j];
                    if (add && TR_LOAD_OK(s.res, rr + j, int(sizeof(T)))) pr[j] = rr[j];
                }
                ptx::fence_proxy_async_smem();
                __syncthreads();
            }
        }
        T *ho = static_cast<T *>(a.h) + row * a.ld_h;
        float h[N][V];
        float2 sums = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if constexpr (VEC) {
                const int lo = column(i, 0);
                uint4 raw = make_uint4(0u, 0u, 0u, 0u), more = raw;
                if (lo < cols) {
                    raw = *reinterpret_cast<const uint4 *>(px + lo);
                    if (add) more = *reinterpret_cast<const uint4 *>(pr + lo);
                }
                Pack<T, V> c = *reinterpret_cast<const Pack<T, V> *>(&raw);
                const Pack<T, V> m = *reinterpret_cast<const Pack<T, V> *>(&more);
                if (add) {
                    float v[V];
#pragma unroll
                    for (int q = 0; q < V; ++q) v[q] = c.get(q) + m.get(q);
                    c.round(v);
                    if (lo < cols) store_chunk<T, V, false>(ho, lo, cols, c, s.h);
                }
#pragma unroll
                for (int q = 0; q < V; ++q) h[i][q] = c.get(q);
            } else {
#pragma unroll
                for (int q = 0; q < V; ++q) {
                    const int j = column(i, q);
                    float v = j < cols ? to_f32(px[j]) : 0.0f;
                    if (add && j < cols) {
                        v = round_to(v + to_f32(pr[j]), T(0.0f));
                        if (TR_STORE_OK(s.h, ho + j, int(sizeof(T)))) put_value(ho + j, v);
                    }
                    h[i][q] = v;
                }
            }
#pragma unroll
            for (int q = 0; q < V; q += 2) sums = __ffma2_rn(make_float2(h[i][q], h[i][q + 1]), make_float2(h[i][q], h[i][q + 1]), sums);
        }
        const float sum = block_sum(sums.x + sums.y, slots[turn]);
        if (t == 0 && ok) {  // past its meeting the block has read this row
            const int64_t next = row + int64_t(stages) * gridDim.x;
            if (next < a.rows) issue(next, stage);
        }
        const float rstd = 1.0f / sqrtf(fmaf(sum, a.inv_cols, a.eps));
        if (t == 0 && a.rstd && TR_STORE_OK(s.rstd, a.rstd + row, 4)) a.rstd[row] = rstd;
        T *yo = static_cast<T *>(a.y) + row * a.ld_y;
        float y[N][V];
#pragma unroll
        for (int i = 0; i < N; ++i) normed<V>(y[i], h[i], rstd, w[i]);
        if constexpr (VEC) {
            int lo[N];
#pragma unroll
            for (int i = 0; i < N; ++i) {
                lo[i] = column(i, 0);
                if (a.y && lo[i] < cols) {
                    Pack<T, V> o;
                    o.round(y[i]);
                    store_chunk<T, V, false>(yo, lo[i], cols, o, s.y);
                }
            }
            if (a.q) quantize_chunks<V, N>(a, row, lo, y, s);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                float m = kFloor;
#pragma unroll
                for (int q = 0; q < V; ++q) {
                    const int j = column(i, q);
                    if (a.y && j < cols && TR_STORE_OK(s.y, yo + j, int(sizeof(T)))) put_value(yo + j, y[i][q]);
                    m = max_abs(m, y[i][q]);
                }
                if (!a.q || column(i, 0) - lane >= cols) continue;
                // One division for both ratios: lane 0 takes the scale.
                const float amax = __uint_as_float(__reduce_max_sync(0xffffffffu, bits_of(m)));
                const float ratio = (lane == 0 ? amax : a.top) / (lane == 0 ? a.top : amax), inv = __shfl_sync(0xffffffffu, ratio, 1);
                if (lane == 0) {
                    float *p = a.scale + int64_t(column(i, 0) >> 7) * a.ld_scale + row;
                    if (TR_STORE_OK(s.scale, p, 4)) *p = ratio;
                }
                uint32_t word[1];
                if (a.e5m2) to_words<true, 4>(word, y[i], inv);
                else to_words<false, 4>(word, y[i], inv);
#pragma unroll
                for (int q = 0; q < V; ++q) {
                    uint8_t *p = a.q + row * a.ld_q + column(i, q);
                    if (column(i, q) < cols && TR_STORE_OK(s.q, p, 1)) *p = uint8_t(word[0] >> (8 * q));
                }
            }
        }
        turn ^= 1;
        if (++stage == stages) {
            stage = 0;
            phase ^= 1;
        }
    }
    if (!ok) {
        atomicExch(&g_fault_flag_rmsnorm, 1u);
        for (int i = 0; i < stages; ++i) {  // no copy may land after the block has gone
            ptx::mbar_wait_bounded(full + i, 0);
            ptx::mbar_wait_bounded(full + i, 1);
        }
    }
}

// Rows that neither holds: one to a block, in two walks, one value to an access.
template <typename T>
__global__ void __launch_bounds__(1024) k_rmsnorm_any(const Rms a) {
    pdl_prologue();
    __shared__ float slots[2][32];
    const RmsSides s = sides_of<T>(a);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int turn = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
        const T *x = static_cast<const T *>(a.x) + row * a.ld_x;
        const T *r = static_cast<const T *>(a.residual) + row * a.ld_residual;
        T *h = static_cast<T *>(a.h) + row * a.ld_h;
        T *y = static_cast<T *>(a.y) + row * a.ld_y;
        float sum[1] = {0.0f};
        for (int64_t j = threadIdx.x; j < a.cols; j += blockDim.x) {
            float v = TR_LOAD_OK(s.x, x + j, int(sizeof(T))) ? to_f32(x[j]) : 0.0f;
            if (a.residual) {
                if (TR_LOAD_OK(s.res, r + j, int(sizeof(T)))) v += to_f32(r[j]);
                v = round_to(v, T(0.0f));
                if (TR_STORE_OK(s.h, h + j, int(sizeof(T)))) put_value(h + j, v);
            }
            sum[0] = fmaf(v, v, sum[0]);
        }
        group_sum<1024, 1>(sum, slots[turn]);
        const float rstd = 1.0f / sqrtf(fmaf(sum[0], a.inv_cols, a.eps));
        if (threadIdx.x == 0 && a.rstd && TR_STORE_OK(s.rstd, a.rstd + row, 4)) a.rstd[row] = rstd;
        const T *from = a.residual ? h : x;
        for (int64_t c0 = int64_t(warp) * 128; c0 < a.cols; c0 += int64_t(blockDim.x) * 4) {
            float v[4];
            uint32_t most = kFloorBits;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int64_t j = c0 + k * 32 + lane;
                v[k] = j < a.cols ? to_f32(from[j]) * rstd * weight(a.gamma, a.w_bf16, j, s.w) : 0.0f;
                if (a.y && j < a.cols && TR_STORE_OK(s.y, y + j, int(sizeof(T)))) put_value(y + j, v[k]);
                most = max(most, bits_of(v[k]));
            }
            if (!a.q) continue;
            const float amax = __uint_as_float(__reduce_max_sync(0xffffffffu, most));
            const float inv = a.top / amax;
            if (lane == 0) {
                float *p = a.scale + (c0 >> 7) * a.ld_scale + row;
                if (TR_STORE_OK(s.scale, p, 4)) *p = amax / a.top;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int64_t j = c0 + k * 32 + lane;
                uint8_t *q = a.q + row * a.ld_q + j;
                if (j < a.cols && TR_STORE_OK(s.q, q, 1)) *q = to_byte(v[k] * inv, a.e5m2);
            }
        }
    }
}

// The transposed 8-bit output, a 128 x 128 tile of h at a time: a thread holds the 8 x 8 values of row group rg
// and column group cg, as the quantizer does.  The last rows of h are the likeliest to be in L2 still, so the tiles
// are walked from the last to the first.  VEC: rows of h on 16-byte boundaries.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256, sizeof(T) == 2 ? 3 : 2) k_rmsnorm_turned(const Rms a) {
    pdl_prologue();
    __shared__ alignas(16) float col_max[8][128];
    __shared__ alignas(16) float col_inv[128];
    __shared__ uint2 turned[128 * 16];
    const T *src = static_cast<const T *>(a.residual ? a.h : a.x);
    const int64_t ld = a.residual ? a.ld_h : a.ld_x;
    [[maybe_unused]] const dbg::Side sh = dbg::side(src, 1, a.rows, a.cols, ld, 0, sizeof(T));
    [[maybe_unused]] const dbg::Side sw = dbg::side(a.gamma, 1, 1, a.cols, a.cols, 0, a.w_bf16 ? 2 : 4);
    [[maybe_unused]] const dbg::Side sd = dbg::side(a.rstd, 1, 1, a.rows, a.rows, 0, 4);
    [[maybe_unused]] const dbg::Side st = dbg::side(a.qt, 1, a.cols, a.rows, a.ld_qt, 0, 1);
    [[maybe_unused]] const dbg::Side su = dbg::side(a.scale_t, 1, (a.rows + 127) / 128, a.cols, a.ld_scale_t, 0, 4);
    const int64_t tiles_r = (a.rows + 127) / 128, tiles_c = (a.cols + 127) / 128;
    const int t = threadIdx.x, lane = t & 31, cg = t & 15, rg = t >> 4, warp = t >> 5;
    for (int64_t at = tiles_r * tiles_c - 1 - int64_t(blockIdx.x); at >= 0; at -= gridDim.x) {
        const int64_t tr = at / tiles_c, tc = at - tr * tiles_c, r0 = tr * 128 + rg * 8, c0 = tc * 128 + cg * 8;
        Pack<T, 16 / int(sizeof(T))> h[8][sizeof(T) / 2];
        constexpr int W = 16 / int(sizeof(T));
        float rstd[8], w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const T *p = src + (r0 + i) * ld;
#pragma unroll
            for (int k = 0; k < int(sizeof(T)) / 2; ++k) {
                if (VEC && r0 + i < a.rows && c0 + (k + 1) * W <= a.cols) {
                    h[i][k] = load_chunk<T, W, false>(p, c0 + k * W, a.cols, sh);
                } else {
                    h[i][k].clear();
                    if (r0 + i < a.rows)
#pragma unroll
                        for (int q = 0; q < W; ++q)
                            if (c0 + k * W + q < a.cols && TR_LOAD_OK(sh, p + c0 + k * W + q, int(sizeof(T)))) h[i][k].set(q, p[c0 + k * W + q]);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            rstd[i] = r0 + i < a.rows && TR_LOAD_OK(sd, a.rstd + r0 + i, 4) ? a.rstd[r0 + i] : 0.0f;
            w[i] = c0 + i < a.cols ? weight(a.gamma, a.w_bf16, c0 + i, sw) : 0.0f;
        }
        // Columns j and j + 1 of row i.
        auto pair = [&](int i, int j) {
            return __fmul2_rn(__fmul2_rn(make_float2(h[i][j / W].get(j % W), h[i][j / W].get(j % W + 1)), make_float2(rstd[i], rstd[i])),
                              make_float2(w[j], w[j + 1]));
        };
        float most[8];
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            most[j] = most[j + 1] = kFloor;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 v = pair(i, j);
                most[j] = max_abs(most[j], v.x);
                most[j + 1] = max_abs(most[j + 1], v.y);
            }
            most[j] = max_abs(most[j], __shfl_xor_sync(0xffffffffu, most[j], 16));
            most[j + 1] = max_abs(most[j + 1], __shfl_xor_sync(0xffffffffu, most[j + 1], 16));
        }
        if (lane < 16) {
            float4 *p = reinterpret_cast<float4 *>(&col_max[warp][cg * 8]);
            p[0] = make_float4(most[0], most[1], most[2], most[3]);
            p[1] = make_float4(most[4], most[5], most[6], most[7]);
        }
        __syncthreads();
        if (t < 128) {
            float amax = kFloor;
#pragma unroll
            for (int k = 0; k < 8; ++k) amax = max_abs(amax, col_max[k][t]);
            col_inv[t] = a.top / amax;
            if (tc * 128 + t < a.cols) {
                float *u = a.scale_t + tr * a.ld_scale_t + tc * 128 + t;
                if (TR_STORE_OK(su, u, 4)) *u = amax / a.top;
            }
        }
        __syncthreads();
        auto turn = [&](auto e5m2) {
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                const float2 inv = *reinterpret_cast<const float2 *>(&col_inv[cg * 8 + j]);
                float2 v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = __fmul2_rn(pair(i, j), inv);
                constexpr __nv_fp8_interpretation_t K = decltype(e5m2)::value ? __NV_E5M2 : __NV_E4M3;
                uint32_t a[4], b[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    a[i] = __nv_cvt_float2_to_fp8x2(make_float2(v[2 * i].x, v[2 * i + 1].x), __NV_SATFINITE, K);
                    b[i] = __nv_cvt_float2_to_fp8x2(make_float2(v[2 * i].y, v[2 * i + 1].y), __NV_SATFINITE, K);
                }
                turned[(cg * 8 + j) * 16 + (rg ^ cg)] = make_uint2(a[0] | a[1] << 16, a[2] | a[3] << 16);
                turned[(cg * 8 + j + 1) * 16 + (rg ^ cg)] = make_uint2(b[0] | b[1] << 16, b[2] | b[3] << 16);
            }
        };
        if (a.e5m2) turn(std::true_type());
        else turn(std::false_type());
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int c = i * 16 + rg;
            const int64_t col = tc * 128 + c;
            if (col < a.cols) store8(a.qt + col * a.ld_qt, tr * 128 + cg * 8, a.rows, turned[c * 16 + (cg ^ (c >> 3))], st);
        }
        __syncthreads();  // the shared words are written anew in the next turn
    }
}

// The ring kernel's launch; cudaErrorNotSupported where a ring of two rows does not fit.
template <typename T>
cudaError_t launch_ring(const Rms &a, bool vec, cudaStream_t stream) {
    if (a.cols > 16384) return cudaErrorNotSupported;
    int threads = 64;
    while (threads * 16 < a.cols) threads *= 2;
    const uint32_t row_bytes = uint32_t((a.cols * int64_t(sizeof(T)) + 30) / 16 * 16), stage_bytes = a.residual ? 2 * row_bytes : row_bytes;
    // 1024 threads to an SM, in as many blocks; fewer where the ring or the rows want it.
    int64_t per_sm = 1024 / threads;
    while (per_sm > 1 && ring_room(per_sm) / stage_bytes < 3) per_sm /= 2;
    const uint32_t fit = ring_room(per_sm) / stage_bytes;
    if (fit < 2) return cudaErrorNotSupported;
    const int stages = int(fit < kMaxStages ? fit : kMaxStages);
    // Five rows to a block, or 160 KB of them, whatever is resident: more blocks than that balance, and a block's end
    // overlaps another's start.  16384 x 8192 bf16 takes 181.6 us with resident blocks that walk all rows, 162.4, 157.5,
    // 155.8 and 172.0 with 4, 8, 16 and 32 times as many (2 rows each); 12289 x 7919 fp32 261.5, 243.0, 236.3, 232.4 and
    // 244.0.  Blocks of neighbouring rows are slower than blocks of every n-th one (fp32 238.9, 16 times).
    const int64_t resident = int64_t(sm_count()) * per_sm, each = 160 * 1024 / stage_bytes > 5 ? 160 * 1024 / stage_bytes : 5;
    int64_t grid = (a.rows + each - 1) / each;
    if (grid < resident) grid = a.rows < resident ? a.rows : resident;
    // Always the most that any call needs.
    const cudaError_t e = vec ? allow_shared<k_rmsnorm_ring<T, true>>(ring_room(1)) : allow_shared<k_rmsnorm_ring<T, false>>(ring_room(1));
    if (e != cudaSuccess) return e;
    return launch_pdl(vec ? k_rmsnorm_ring<T, true> : k_rmsnorm_ring<T, false>, dim3(unsigned(grid)),
                      dim3(unsigned(threads)), size_t(stages) * stage_bytes, stream, a, stages, row_bytes);
}

template <typename T>
cudaError_t launch_rows(const Rms &a, cudaStream_t stream) {
    constexpr int V = 16 / int(sizeof(T)), es = int(sizeof(T));
    const bool vec = a.cols % V == 0 && side_aligned16(a.x, a.ld_x, 0, 1, es) && (!a.y || side_aligned16(a.y, a.ld_y, 0, 1, es)) &&
                     (!a.residual || (side_aligned16(a.residual, a.ld_residual, 0, 1, es) && side_aligned16(a.h, a.ld_h, 0, 1, es)));
    const int64_t chunks = a.cols / V, resident = sm_count();
    if (vec && (reinterpret_cast<uintptr_t>(a.gamma) & 15u) == 0) {
        auto run = [&](auto kern, int threads, int rows_per_block, int64_t per_sm) {
            const int64_t want = (a.rows + rows_per_block - 1) / rows_per_block, most = resident * per_sm;
            return launch_pdl(kern, dim3(unsigned(want < most ? want : most)), dim3(unsigned(threads)), 0, stream, a);
        };
        if (chunks <= 128) return run(k_rmsnorm_held<T, 32, 4>, 128, 4, 8);
        if (a.rows <= 2 * resident) {
            if (chunks <= 256) return run(k_rmsnorm_held<T, 256, 1>, 256, 1, 4);
            if (chunks <= 1024) return run(k_rmsnorm_held<T, 1024, 1>, 1024, 1, 1);
            if (chunks <= 2048) return run(k_rmsnorm_held<T, 1024, 2>, 1024, 1, 1);
        }
    }
    const cudaError_t e = launch_ring<T>(a, vec, stream);
    if (e != cudaErrorNotSupported) return e;
    const int64_t most = int64_t(1) << 30;
    return launch_pdl(k_rmsnorm_any<T>, dim3(unsigned(a.rows < most ? a.rows : most)), dim3(1024), 0, stream, a);
}

template <typename T>
cudaError_t launch_typed(const Rms &a, cudaStream_t stream) {
    const cudaError_t e = launch_rows<T>(a, stream);
    if (e != cudaSuccess || !a.qt) return e;
    const int64_t tiles = ((a.rows + 127) / 128) * ((a.cols + 127) / 128), most = int64_t(1) << 30;
    const dim3 grid(unsigned(tiles < most ? tiles : most));
    const bool vec = a.residual ? side_aligned16(a.h, a.ld_h, 0, 1, sizeof(T)) : side_aligned16(a.x, a.ld_x, 0, 1, sizeof(T));
    return vec ? launch_pdl(k_rmsnorm_turned<T, true>, grid, dim3(256), 0, stream, a)
               : launch_pdl(k_rmsnorm_turned<T, false>, grid, dim3(256), 0, stream, a);
}

}  // namespace

TR_WAIT_UNIT(rmsnorm)

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

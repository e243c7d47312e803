// Root-mean-square norm with the residual's addition: h = x + residual, and
// y = h * rstd * gamma with rstd = 1 / sqrt(sum(h^2) / n + eps), as rows of h's type and in
// 8 bits with a scale for each block of 128, by rows and transposed.
//
// Bound by memory: x and residual are read once, h, y, q and qt written once.  The statistics are held in 32 bits, y is
// rounded once, and the 8-bit values come from y in 32 bits, not from its rounded form.  A row stays on the chip between
// its two walks (registers, or shared memory that bulk copies fill rows ahead); the transposed 8-bit output, whose blocks
// of 128 rows need every row's rstd, takes a second launch that reads h once more.  Device time, and the share of the
// copy rate on the bytes above:
//   1 x 8192 bf16 3 us; 16384 x 8192 bf16 157 us (101%), without a residual 87 (91%); 12289 x 7919 fp32 229-240 (96-100%)
//   8 bits, 16384 x 8192 bf16: rows 146 us (95%), both ways 220 (73%: h's second read is 25% more bytes)
//   4000 x 20000 bf16 121 us (78%), rows of 20001 values 486 (19%)
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
// The largest magnitude of three; a NaN wins.
__device__ __forceinline__ float max_abs(float a, float b, float c) {
    float m;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(a), "f"(b), "f"(c));
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
        for (int q = 0; q < V; q += 2) m[n] = max_abs(m[n], y[n][q], y[n][q + 1]);
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
        const float rstd = __frsqrt_rn(fmaf(sum[0], a.inv_cols, a.eps));
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
    const int64_t first = blockIdx.x, step = gridDim.x;
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
        for (int i = 0; i < stages && first + i * step < a.rows; ++i) issue(first + i * step, i);
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
    for (int64_t row = first; row < a.rows; row += step) {
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
            const int64_t next = row + stages * step;
            if (next < a.rows) issue(next, stage);
        }
        const float rstd = __frsqrt_rn(fmaf(sum, a.inv_cols, a.eps));
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
                    if (q % 2) m = max_abs(m, y[i][q - 1], y[i][q]);
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

// Longer rows on 16-byte boundaries: one to a block, in two walks, the second of which finds h in L2.  4000 x 20000 bf16
// 121 us, 468 with k_rmsnorm_any; 4096 x 16384 fp32 178 (89% of the copy rate).
constexpr int kWideThreads = 512;
template <typename T>
__global__ void __launch_bounds__(kWideThreads, 3) k_rmsnorm_wide(const Rms a) {
    pdl_prologue();
    constexpr int V = 16 / int(sizeof(T));
    __shared__ float slots[2][32];
    const RmsSides s = sides_of<T>(a);
    const int64_t first = int64_t(threadIdx.x & ~31) * V, step = kWideThreads * V;  // columns of the warp, the lane's among them
    const int own = (threadIdx.x & 31) * V;
    int turn = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
        const T *x = static_cast<const T *>(a.x) + row * a.ld_x;
        const T *r = static_cast<const T *>(a.residual) + row * a.ld_residual;
        T *h = static_cast<T *>(a.h) + row * a.ld_h;
        T *y = static_cast<T *>(a.y) + row * a.ld_y;
        float sum[1] = {0.0f};
#pragma unroll 2
        for (int64_t c = first; c < a.cols; c += step) {
            const int64_t lo = c + own;
            Pack<T, V> p = load_chunk<T, V, false>(x, lo, a.cols, s.x);
            if (a.residual) {
                const Pack<T, V> o = load_chunk<T, V, false>(r, lo, a.cols, s.res);
                float v[V];
#pragma unroll
                for (int q = 0; q < V; ++q) v[q] = p.get(q) + o.get(q);
                p.round(v);
                if (lo < a.cols) store_chunk<T, V, false>(h, lo, a.cols, p, s.h);
            }
#pragma unroll
            for (int q = 0; q < V; ++q) sum[0] = fmaf(p.get(q), p.get(q), sum[0]);
        }
        group_sum<kWideThreads, 1>(sum, slots[turn]);
        const float rstd = __frsqrt_rn(fmaf(sum[0], a.inv_cols, a.eps));
        if (threadIdx.x == 0 && a.rstd && TR_STORE_OK(s.rstd, a.rstd + row, 4)) a.rstd[row] = rstd;
        const T *from = a.residual ? h : x;  // this thread's own values
#pragma unroll 2
        for (int64_t c = first; c < a.cols; c += step) {
            const int64_t lo = c + own;
            float v[V], w[V], n[1][V];
            const Pack<T, V> p = load_chunk<T, V, false>(from, lo, a.cols, a.residual ? s.h : s.x);
#pragma unroll
            for (int q = 0; q < V; ++q) {
                v[q] = p.get(q);
                w[q] = 0.0f;
            }
            if (lo < a.cols) load_weights<V>(a.gamma, a.w_bf16, lo, w, s.w);
            normed<V>(n[0], v, rstd, w);
            if (a.y && lo < a.cols) {
                Pack<T, V> o;
                o.round(n[0]);
                store_chunk<T, V, false>(y, lo, a.cols, o, s.y);
            }
            const int at[1] = {int(lo)};
            if (a.q) quantize_chunks<V, 1>(a, row, at, n, s);
        }
    }
}

// Rows that none of them takes: one to a block, in two walks, one value to an access.
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
        const float rstd = __frsqrt_rn(fmaf(sum[0], a.inv_cols, a.eps));
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

// Four neighbouring values of a row.
template <typename T>
struct Quad;
template <>
struct Quad<__nv_bfloat16> {
    uint32_t w[2];
    __device__ __forceinline__ void clear() { w[0] = w[1] = 0u; }
    __device__ __forceinline__ void set(int q, __nv_bfloat16 v) { w[q >> 1] |= uint32_t(__bfloat16_as_ushort(v)) << (q & 1 ? 16 : 0); }
    __device__ __forceinline__ float get(int q) const { return __uint_as_float(q & 1 ? w[q >> 1] & 0xffff0000u : w[q >> 1] << 16); }
    __device__ __forceinline__ void held(const void *p) {  // in shared memory
        const uint2 v = *static_cast<const uint2 *>(p);
        w[0] = v.x;
        w[1] = v.y;
    }
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) {
        const uint2 v = __ldcs(reinterpret_cast<const uint2 *>(p));
        w[0] = v.x;
        w[1] = v.y;
    }
};
template <>
struct Quad<float> {
    float e[4];
    __device__ __forceinline__ void clear() { e[0] = e[1] = e[2] = e[3] = 0.0f; }
    __device__ __forceinline__ void set(int q, float v) { e[q] = v; }
    __device__ __forceinline__ float get(int q) const { return e[q]; }
    __device__ __forceinline__ void held(const void *p) {
        const float4 v = *static_cast<const float4 *>(p);
        e[0] = v.x;
        e[1] = v.y;
        e[2] = v.z;
        e[3] = v.w;
    }
    __device__ __forceinline__ void load(const float *p) {
        const float4 v = __ldcs(reinterpret_cast<const float4 *>(p));
        e[0] = v.x;
        e[1] = v.y;
        e[2] = v.z;
        e[3] = v.w;
    }
};

constexpr int kTurners = 512;  // threads to a tile
struct TurnSpace {
    float most[16][128];
    float inv[128], rstd[128], w[128];
    uint2 turned[128 * 16];
};

// The transposed 8-bit output after the rows, a 128 x 128 tile of h at a time: a thread holds 8 rows (group rg, its
// warp) of 4 columns (group cg, its lane), as u = h * rstd for both walks over it.  The bytes go through shared memory in
// slots of 8, slot XOR column group.  AHEAD: the next tile's rows, on 16-byte boundaries, are copied to shared memory
// meanwhile (a block meets four times a tile, and two blocks to an SM do not cover for one another: 16384 x 8192
// bf16 takes 88 us without); else they come straight from memory, VEC in one access to four values.  The last rows
// of h are the likeliest to be in L2 still, so the tiles are walked from the last to the first.
//
// With these tiles in the same launch as the rows, each waiting for its rows' rstd, so that h comes from L2, 16384 x
// 8192 bf16 took 259 us, 234 with this kernel's first form after the rows'.
template <typename T, bool VEC, bool AHEAD>
__global__ void __launch_bounds__(kTurners, 2) k_rmsnorm_turned(const Rms a) {
    pdl_prologue();
    __shared__ alignas(16) TurnSpace m;
    extern __shared__ uint4 ring4[];  // AHEAD: two tiles
    const T *src = static_cast<const T *>(a.residual ? a.h : a.x);
    const int64_t ld = a.residual ? a.ld_h : a.ld_x;
    [[maybe_unused]] const dbg::Side sh = dbg::side(src, 1, a.rows, a.cols, ld, 0, sizeof(T));
    [[maybe_unused]] const dbg::Side sw = dbg::side(a.gamma, 1, 1, a.cols, a.cols, 0, a.w_bf16 ? 2 : 4);
    [[maybe_unused]] const dbg::Side sd = dbg::side(a.rstd, 1, 1, a.rows, a.rows, 0, 4);
    [[maybe_unused]] const dbg::Side st = dbg::side(a.qt, 1, a.cols, a.rows, a.ld_qt, 0, 1);
    [[maybe_unused]] const dbg::Side su = dbg::side(a.scale_t, 1, (a.rows + 127) / 128, a.cols, a.ld_scale_t, 0, 4);
    const int t = threadIdx.x, cg = t & 31, rg = t >> 5;
    // Tiles counted in 32 bits: a 64-bit division would be a hundred instructions to each thread.
    const uint32_t tiles_c = uint32_t((a.cols + 127) / 128), tiles = uint32_t((a.rows + 127) / 128) * tiles_c;
    constexpr int kChunks = 128 * int(sizeof(T)) / 16, kRow = 128 * int(sizeof(T));  // of a tile's row: granules, bytes
    // What tile `at` needs: rstd of its rows and the weights of its columns, one to each of 256 threads, and its rows.
    auto number = [&](uint32_t at) {
        const int64_t row = int64_t(at / tiles_c) * 128 + t, col = int64_t(at % tiles_c) * 128 + t - 128;
        if (t < 128) return row < a.rows && TR_LOAD_OK(sd, a.rstd + row, 4) ? a.rstd[row] : 0.0f;
        return t < 256 && col < a.cols ? weight(a.gamma, a.w_bf16, col, sw) : 0.0f;
    };
    auto copy = [&](uint32_t at, int buffer) {
        if constexpr (AHEAD) {
            uint8_t *to = reinterpret_cast<uint8_t *>(ring4) + size_t(buffer) * 128 * kRow;
#pragma unroll
            for (int k = 0; k < 128 * kChunks / kTurners; ++k) {
                const int id = t + k * kTurners, r = id / kChunks, c = id % kChunks;
                const int64_t row = int64_t(at / tiles_c) * 128 + r, col = int64_t(at % tiles_c) * 128 + c * (16 / int(sizeof(T)));
                uint8_t *dst = to + r * kRow + c * 16;
                const T *p = src + row * ld + col;
                if (row < a.rows && col < a.cols && TR_LOAD_OK(sh, p, 16)) ptx::cp_async_16(dst, p);
                else *reinterpret_cast<uint4 *>(dst) = make_uint4(0u, 0u, 0u, 0u);
            }
            ptx::cp_async_commit();
        }
    };
    uint32_t left = blockIdx.x;  // tiles are counted from the end
    if (left >= tiles) return;
    float next = number(tiles - 1 - left);
    copy(tiles - 1 - left, 0);
    for (int buffer = 0; left < tiles; left += gridDim.x, buffer ^= 1) {
        const uint32_t at = tiles - 1 - left;
        const int64_t tr = at / tiles_c, tc = at % tiles_c, r0 = tr * 128 + rg * 8, c0 = tc * 128 + cg * 4;
        const bool whole = VEC && tr * 128 + 128 <= a.rows && tc * 128 + 128 <= a.cols;
        if (t < 128) m.rstd[t] = next;
        else if (t < 256) m.w[t - 128] = next;
        const bool more = tiles - left > gridDim.x;
        if (more) {
            next = number(at - gridDim.x);
            copy(at - gridDim.x, buffer ^ 1);
        }
        Quad<T> h[8];
        if constexpr (AHEAD) {
            if (more) ptx::cp_async_wait<1>();
            else ptx::cp_async_wait<0>();
            __syncthreads();
            const uint8_t *from = reinterpret_cast<const uint8_t *>(ring4) + size_t(buffer) * 128 * kRow;
#pragma unroll
            for (int i = 0; i < 8; ++i) h[i].held(from + (rg * 8 + i) * kRow + cg * 4 * int(sizeof(T)));
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const T *p = src + (r0 + i) * ld + c0;
                h[i].clear();
                if (VEC && (whole || (r0 + i < a.rows && c0 + 4 <= a.cols))) {
                    if (TR_LOAD_OK(sh, p, int(4 * sizeof(T)))) h[i].load(p);
                } else if (r0 + i < a.rows) {
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        if (c0 + q < a.cols && TR_LOAD_OK(sh, p + q, int(sizeof(T)))) h[i].set(q, p[q]);
                }
            }
            __syncthreads();
        }
        float2 u[8][2];
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float rstd = m.rstd[rg * 8 + i];
                u[i][j] = make_float2(h[i].get(2 * j) * rstd, h[i].get(2 * j + 1) * rstd);
            }
        const float4 w4 = *reinterpret_cast<const float4 *>(&m.w[cg * 4]);
        const float2 w[2] = {make_float2(w4.x, w4.y), make_float2(w4.z, w4.w)};
        float2 most[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            most[j] = make_float2(kFloor, kFloor);
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                const float2 v = __fmul2_rn(u[i][j], w[j]), x = __fmul2_rn(u[i + 1][j], w[j]);
                most[j].x = max_abs(most[j].x, v.x, x.x);
                most[j].y = max_abs(most[j].y, v.y, x.y);
            }
        }
        *reinterpret_cast<float4 *>(&m.most[rg][cg * 4]) = make_float4(most[0].x, most[0].y, most[1].x, most[1].y);
        __syncthreads();
        if (t < 128) {
            float amax = kFloor;
#pragma unroll
            for (int k = 0; k < 16; k += 2) amax = max_abs(amax, m.most[k][t], m.most[k + 1][t]);
            m.inv[t] = a.top / amax;
            if (tc * 128 + t < a.cols) {
                float *p = a.scale_t + tr * a.ld_scale_t + tc * 128 + t;
                if (TR_STORE_OK(su, p, 4)) *p = amax / a.top;
            }
        }
        __syncthreads();
        auto bytes = [&](auto e5m2) {
            constexpr __nv_fp8_interpretation_t K = decltype(e5m2)::value ? __NV_E5M2 : __NV_E4M3;
            const float4 inv4 = *reinterpret_cast<const float4 *>(&m.inv[cg * 4]);
            const float2 inv[2] = {make_float2(inv4.x, inv4.y), make_float2(inv4.z, inv4.w)};
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                uint32_t p[4], q[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 x = __fmul2_rn(__fmul2_rn(u[2 * i][j], w[j]), inv[j]), v = __fmul2_rn(__fmul2_rn(u[2 * i + 1][j], w[j]), inv[j]);
                    p[i] = __nv_cvt_float2_to_fp8x2(make_float2(x.x, v.x), __NV_SATFINITE, K);
                    q[i] = __nv_cvt_float2_to_fp8x2(make_float2(x.y, v.y), __NV_SATFINITE, K);
                }
                uint2 *slot = m.turned + (cg * 4 + 2 * j) * 16 + (rg ^ (cg & 15));
                slot[0] = make_uint2(p[0] | p[1] << 16, p[2] | p[3] << 16);
                slot[16] = make_uint2(q[0] | q[1] << 16, q[2] | q[3] << 16);
            }
        };
        if (a.e5m2) bytes(std::true_type());
        else bytes(std::false_type());
        __syncthreads();
        const int r = t & 15;
        uint8_t *p = a.qt + (tc * 128 + (t >> 4)) * a.ld_qt;
#pragma unroll
        for (int i = 0; i < 4; ++i, p += 32 * a.ld_qt) {
            const int c = i * 32 + (t >> 4);
            const uint2 v = m.turned[c * 16 + (r ^ (c >> 2 & 15))];
            if (whole) {
                if (TR_STORE_OK(st, p + tr * 128 + r * 8, 8)) *reinterpret_cast<uint2 *>(p + tr * 128 + r * 8) = v;
            } else if (tc * 128 + c < a.cols) {
                store8(p, tr * 128 + r * 8, a.rows, v, st);
            }
        }
        // The next turn writes rstd and w (read before two meetings) at once, everything else past its first meeting.
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
    if (grid > int64_t(1) << 30) grid = int64_t(1) << 30;
    // Always the most that any call needs.
    const cudaError_t e = vec ? allow_shared<k_rmsnorm_ring<T, true>>(ring_room(1)) : allow_shared<k_rmsnorm_ring<T, false>>(ring_room(1));
    if (e != cudaSuccess) return e;
    return launch_pdl(vec ? k_rmsnorm_ring<T, true> : k_rmsnorm_ring<T, false>, dim3(unsigned(grid)),
                      dim3(unsigned(threads)), size_t(stages) * stage_bytes, stream, a, stages, row_bytes);
}

template <typename T>
bool rows_aligned(const Rms &a) {
    constexpr int V = 16 / int(sizeof(T)), es = int(sizeof(T));
    return a.cols % V == 0 && side_aligned16(a.x, a.ld_x, 0, 1, es) && (!a.y || side_aligned16(a.y, a.ld_y, 0, 1, es)) &&
           (!a.residual || (side_aligned16(a.residual, a.ld_residual, 0, 1, es) && side_aligned16(a.h, a.ld_h, 0, 1, es)));
}

template <typename T>
cudaError_t launch_rows(const Rms &a, cudaStream_t stream) {
    constexpr int V = 16 / int(sizeof(T));
    const bool vec = rows_aligned<T>(a);
    const int64_t chunks = a.cols / V, resident = sm_count();
    if (vec && (reinterpret_cast<uintptr_t>(a.gamma) & 15u) == 0) {
        auto run = [&](auto kern, int threads, int rows_per_block, int64_t per_sm) {
            const int64_t want = (a.rows + rows_per_block - 1) / rows_per_block, most = resident * per_sm;
            return launch_pdl(kern, dim3(unsigned(want < most ? want : most)), dim3(unsigned(threads)), 0, stream, a);
        };
        // A warp to a row.  Rows of one chunk to a lane, 262144 x 128 bf16 with a residual: 135 us with four chunks' code and
        // resident blocks, 74 with one chunk's, 62 with four times as many blocks as are resident.
        if (chunks <= 32) return run(k_rmsnorm_held<T, 32, 1>, 128, 4, 48);
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
    const dim3 grid(unsigned(a.rows < most ? a.rows : most));
    if (vec && a.cols <= int64_t(1) << 30 && (reinterpret_cast<uintptr_t>(a.gamma) & 15u) == 0)  // columns in 32 bits
        return launch_pdl(k_rmsnorm_wide<T>, grid, dim3(kWideThreads), 0, stream, a);
    return launch_pdl(k_rmsnorm_any<T>, grid, dim3(1024), 0, stream, a);
}

template <typename T>
cudaError_t launch_typed(const Rms &a, cudaStream_t stream) {
    const cudaError_t e = launch_rows<T>(a, stream);
    if (e != cudaSuccess || !a.qt) return e;
    const int64_t tiles = ((a.rows + 127) / 128) * ((a.cols + 127) / 128), resident = 2 * int64_t(sm_count());
    if (tiles > 0x7fffffffll) return cudaErrorInvalidValue;
    const dim3 grid(unsigned(tiles < resident ? tiles : resident));
    constexpr int V = 16 / int(sizeof(T));
    const bool vec = a.cols % V == 0 && (a.residual ? side_aligned16(a.h, a.ld_h, 0, 1, sizeof(T)) : side_aligned16(a.x, a.ld_x, 0, 1, sizeof(T)));
    if constexpr (sizeof(T) == 2) {
        if (vec) {
            constexpr size_t two = 2 * 128 * 128 * sizeof(T);
            const cudaError_t allowed = allow_shared<k_rmsnorm_turned<T, true, true>>(two);
            return allowed != cudaSuccess ? allowed : launch_pdl(k_rmsnorm_turned<T, true, true>, grid, dim3(kTurners), two, stream, a);
        }
    }
    return vec ? launch_pdl(k_rmsnorm_turned<T, true, false>, grid, dim3(kTurners), 0, stream, a)
               : launch_pdl(k_rmsnorm_turned<T, false, false>, grid, dim3(kTurners), 0, stream, a);
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

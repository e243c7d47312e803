// Layer norm, backward: the input's gradient along the rows, the weight's and
// the bias's down the columns.  With u = (x - mean) * rstd and g = dy * gamma,
//
//   dx = rstd * (g - sum(g)/n - u * sum(g u)/n),  dgamma = sum_rows dy u,  dbeta = sum_rows dy
//
// Bound by memory: one read of x and dy, one write of dx.  The column sums come from
// the same read (k_ln_backward); two kernels, one along the rows and one down the
// columns, take five passes over the matrices instead of three and serve the rows
// that the ring below does not hold: over 16384 columns, and fp32 over 11568, where two
// rows of x and dy (16 bytes to a column) beside the weights (4) pass its 231424 bytes.
//
// Measured on one GB300 (share of the measured copy rate, 6771 GB/s), both kernels:
//   16384 x 8192 bf16   139 us, 5.8 TB/s (86%); row sums and column sums apart: 574 us
//   12289 x 7919 fp32   178 us, 6.6 TB/s (97%)  (rows off 16-byte boundaries)
//   32768 x 4096 bf16   136 us, 5.9 TB/s (87%)
//   16384 x 8192 fp32   266 us, 6.0 TB/s (89%): three rows in flight fill the ring
//   8192 x 9000, 12288, 16384 bf16   257, 283, 338 us: 1.7, 2.1, 2.4 TB/s (values read twice
//                                    from the ring, weights from shared memory)
//   8192 x 11568 / 11572 fp32        274 / 481 us, 4.2 / 2.4 TB/s: the last that the ring holds, and past it
//   8192 x 20480 bf16                713 us, 1.4 TB/s
//   256 x 1024 bf16       9 us: two launches
// The bf16 rows are bound by what a row costs beside its bytes: 0.48 instructions
// a cycle and scheduler, and a meeting of the block per row.
#include "launch.cuh"
#include "ptx.cuh"
#include "row_chunk.cuh"
#include "row_ring.cuh"
#include "tr_internal.h"
#include "wait_selftest.cuh"

namespace tr {

// Set when a bounded in-kernel wait ran out; read and cleared by the host.
__device__ unsigned g_fault_flag_layernorm = 0;

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

// Sums of two values over the block, in every thread; `slot` holds 32 pairs.
__device__ __forceinline__ float2 block_sum2(float s1, float s2, float2 *slot) {
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    // The lanes' halves take one value each, so the two cost six shuffles.
    auto both = [&](float a, float b) {
        const float got = __shfl_xor_sync(0xffffffffu, lane & 16 ? a : b, 16);
        float v = (lane & 16 ? b : a) + got;
#pragma unroll
        for (int o = 8; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        return v;
    };
    float v = both(s1, s2);
    if ((lane & 15) == 0) (lane ? slot[threadIdx.x >> 5].y : slot[threadIdx.x >> 5].x) = v;
    __syncthreads();
    const float2 p = lane < warps ? slot[lane] : make_float2(0.0f, 0.0f);
    v = both(p.x, p.y);
    return make_float2(__shfl_sync(0xffffffffu, v, 0), __shfl_sync(0xffffffffu, v, 16));
}

// The rows' gradients and the columns' sums from one read of x and dy.  A
// resident block walks rows; bulk copies keep a ring of its next rows in
// flight, so no register holds loaded data and any alignment reads whole
// granules.  A thread owns the same 16 columns of every row and sums their dy*u
// and dy in registers (two columns to an instruction); the blocks' sums are
// joined by k_ln_join.  VEC: columns in 16-byte chunks, every row on a 16-byte
// boundary; else one column at a time, neighbouring threads on neighbouring
// columns.  KEEP (up to 8192 columns): 512 threads to an SM, with a row's u and g
// in registers between its two walks; else 1024, which read them from the ring
// again, and the weights from shared memory.
template <typename T, bool KEEP, bool VEC>
__global__ void __launch_bounds__(KEEP ? 512 : 1024, 1)
k_ln_backward(const Bwd a, int stages, uint32_t row_bytes) {
    constexpr int V = VEC ? 16 / int(sizeof(T)) : 1;
    constexpr int P = 8;  // pairs of columns to a thread
    extern __shared__ uint4 ring4[];
    __shared__ uint64_t full[kMaxStages];
    __shared__ float2 slots[2][32];
    uint8_t *ring = reinterpret_cast<uint8_t *>(ring4);
    float *gammas = reinterpret_cast<float *>(ring + size_t(stages) * 2 * row_bytes);  // without KEEP
    [[maybe_unused]] const dbg::Side sd = dbg::side(a.dy, 1, a.rows, a.cols, a.ld_dy, 0, sizeof(T));
    [[maybe_unused]] const dbg::Side sx = dbg::side(a.x, 1, a.rows, a.cols, a.ld_x, 0, sizeof(T));
    [[maybe_unused]] const dbg::Side so = dbg::side(a.dx, 1, a.rows, a.cols, a.ld_dx, 0, sizeof(T));
    [[maybe_unused]] const dbg::Side sw = dbg::side(a.gamma, 1, 1, a.cols, a.cols, 0, a.w_bf16 ? 2 : 4);
    [[maybe_unused]] const dbg::Side sm = dbg::side(a.mean, 1, 1, a.rows, a.rows, 0, 4);
    [[maybe_unused]] const dbg::Side sr = dbg::side(a.rstd, 1, 1, a.rows, a.rows, 0, 4);
    [[maybe_unused]] const dbg::Side sp = dbg::side(a.part, 1, 2 * a.parts, a.cols, a.cols, 0, 4);
    const int t = threadIdx.x, nt = blockDim.x, cols = int(a.cols);
    if (t == 0) {
        for (int i = 0; i < stages; ++i) ptx::mbar_init(full + i, 1);
        ptx::fence_barrier_init();
    }
    __syncthreads();
    pdl_prologue();
    auto issue = [&](int64_t row, int stage) {  // one thread
        const Granules gx = granules<T>(a.x, a.rows, a.cols, a.ld_x, row);
        const Granules gd = granules<T>(a.dy, a.rows, a.cols, a.ld_dy, row);
        uint8_t *at = ring + size_t(stage) * 2 * row_bytes;
        if (!gx.inside || !gd.inside) {  // the block copies that row itself
            ptx::mbar_arrive(full + stage);
            return;
        }
        ptx::mbar_arrive_expect_tx(full + stage, gx.bytes + gd.bytes);
        ptx::bulk_load(at, gx.src, gx.bytes, full + stage);
        ptx::bulk_load(at + row_bytes, gd.src, gd.bytes, full + stage);
    };
    if (t == 0)
        for (int i = 0; i < stages && blockIdx.x + int64_t(i) * gridDim.x < a.rows; ++i)
            issue(blockIdx.x + int64_t(i) * gridDim.x, i);
    // Column of the thread's value e.
    auto column = [&](int e) { return (t + e / V * nt) * V + e % V; };
    // Piece i of its values of a row in shared memory (a chunk, or two single columns),
    // zeros past the row's end.
    constexpr int Q = V < 2 ? 1 : V / 2;  // pairs to a piece
    auto piece = [&](const T *p, int i, float2 (&v)[Q]) {
        if constexpr (VEC) {
            const int j = column(i * V);
            uint4 raw = make_uint4(0u, 0u, 0u, 0u);
            if (j < cols) raw = *reinterpret_cast<const uint4 *>(p + j);
            const Pack<T, V> &c = *reinterpret_cast<const Pack<T, V> *>(&raw);
#pragma unroll
            for (int q = 0; q < Q; ++q) v[q] = make_float2(c.get(2 * q), c.get(2 * q + 1));
        } else {
            const int j0 = column(2 * i), j1 = column(2 * i + 1);
            v[0] = make_float2(j0 < cols ? to_f32(p[j0]) : 0.0f, j1 < cols ? to_f32(p[j1]) : 0.0f);
        }
    };
    auto kept = [&](int j) {
        return j < cols ? weight(a.gamma, a.w_bf16, j, sw) : 0.0f;
    };
    float2 w[KEEP ? P : 1], dg[P], db[P];
#pragma unroll
    for (int k = 0; k < P; ++k) {
        dg[k] = db[k] = make_float2(0.0f, 0.0f);
        if (KEEP) w[KEEP ? k : 0] = make_float2(kept(column(2 * k)), kept(column(2 * k + 1)));
    }
    if (!KEEP) {
        for (int j = t; j < cols; j += nt) gammas[j] = kept(j);
        __syncthreads();
    }
    auto shared_weights = [&](int k) {
        const int j0 = column(2 * k), j1 = column(2 * k + 1);
        return make_float2(j0 < cols ? gammas[j0] : 0.0f, j1 < cols ? gammas[j1] : 0.0f);
    };
    const float inv_cols = 1.0f / float(cols);
    auto stat = [&](const float *p, int64_t row, [[maybe_unused]] const dbg::Side &s) {
        return row < a.rows && TR_LOAD_OK(s, p + row, 4) ? p[row] : 0.0f;
    };
    float mean_next = stat(a.mean, blockIdx.x, sm), rstd_next = stat(a.rstd, blockIdx.x, sr);
    bool ok = true;
    int stage = 0, turn = 0;
    uint32_t phase = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const float mean = mean_next, rstd = rstd_next;
        mean_next = stat(a.mean, row + gridDim.x, sm);
        rstd_next = stat(a.rstd, row + gridDim.x, sr);
        if (ok) ok = ptx::mbar_wait_bounded(full + stage, phase);
        uint8_t *at = ring + size_t(stage) * 2 * row_bytes;
        T *px = reinterpret_cast<T *>(at), *pd = reinterpret_cast<T *>(at + row_bytes);
        if constexpr (!VEC) {
            const Granules gx = granules<T>(a.x, a.rows, a.cols, a.ld_x, row);
            const Granules gd = granules<T>(a.dy, a.rows, a.cols, a.ld_dy, row);
            px = reinterpret_cast<T *>(at + gx.shift);
            pd = reinterpret_cast<T *>(at + row_bytes + gd.shift);
            if (!gx.inside || !gd.inside) {
                const T *xr = static_cast<const T *>(a.x) + row * a.ld_x;
                const T *dr = static_cast<const T *>(a.dy) + row * a.ld_dy;
                for (int j = t; j < cols; j += nt) {
                    if (TR_LOAD_OK(sx, xr + j, int(sizeof(T)))) px[j] = xr[j];
                    if (TR_LOAD_OK(sd, dr + j, int(sizeof(T)))) pd[j] = dr[j];
                }
                ptx::fence_proxy_async_smem();
                __syncthreads();
            }
        }
        const float2 minus_mean = make_float2(-mean, -mean), rstd2 = make_float2(rstd, rstd);
        float2 u[KEEP ? P : 1], g[KEEP ? P : 1], s1 = make_float2(0.0f, 0.0f), s2 = s1;
#pragma unroll
        for (int i = 0; i < P / Q; ++i) {
            float2 x2[Q], d2[Q];
            piece(px, i, x2);
            piece(pd, i, d2);
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                const int k = i * Q + q;
                const float2 uk = __fmul2_rn(__fadd2_rn(x2[q], minus_mean), rstd2);
                const float2 gk = __fmul2_rn(d2[q], KEEP ? w[KEEP ? k : 0] : shared_weights(k));
                dg[k] = __ffma2_rn(d2[q], uk, dg[k]);
                db[k] = __fadd2_rn(db[k], d2[q]);
                s1 = __fadd2_rn(s1, gk);
                s2 = __ffma2_rn(gk, uk, s2);
                if (KEEP) {
                    u[KEEP ? k : 0] = uk;
                    g[KEEP ? k : 0] = gk;
                }
            }
        }
        const float2 s = block_sum2(s1.x + s1.y, s2.x + s2.y, slots[turn]);
        // Past its meeting the block has read this row (KEEP), or left the last one.
        if (t == 0 && ok && (KEEP || row != blockIdx.x)) {
            const int64_t next = row + int64_t(KEEP ? stages : stages - 1) * gridDim.x;
            if (next < a.rows) issue(next, KEEP ? stage : stage == 0 ? stages - 1 : stage - 1);
        }
        const float2 minus_c1 = make_float2(-s.x * inv_cols, -s.x * inv_cols);
        const float2 minus_c2 = make_float2(-s.y * inv_cols, -s.y * inv_cols);
        T *out = static_cast<T *>(a.dx) + row * a.ld_dx;
        float v[2 * P];
#pragma unroll
        for (int i = 0; i < P / Q; ++i) {
            float2 x2[Q], d2[Q];
            if (!KEEP) {
                piece(px, i, x2);
                piece(pd, i, d2);
            }
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                const int k = i * Q + q;
                float2 uk, gk;
                if (KEEP) {
                    uk = u[KEEP ? k : 0];
                    gk = g[KEEP ? k : 0];
                } else {
                    uk = __fmul2_rn(__fadd2_rn(x2[q], minus_mean), rstd2);
                    gk = __fmul2_rn(d2[q], shared_weights(k));
                }
                const float2 r = __fmul2_rn(rstd2, __ffma2_rn(uk, minus_c2, __fadd2_rn(gk, minus_c1)));
                v[2 * k] = r.x;
                v[2 * k + 1] = r.y;
            }
        }
#pragma unroll
        for (int i = 0; i < 2 * P / V; ++i) {
            if (column(i * V) >= cols) continue;
            Pack<T, V> o;
            float whole[V];
#pragma unroll
            for (int q = 0; q < V; ++q) whole[q] = v[i * V + q];
            o.round(whole);
            store_chunk<T, V, false>(out, column(i * V), cols, o, so);
        }
        turn ^= 1;
        if (++stage == stages) {
            stage = 0;
            phase ^= 1;
        }
    }
    if (!ok) {
        atomicExch(&g_fault_flag_layernorm, 1u);
        for (int i = 0; i < stages; ++i) {  // no copy may land after the block has gone
            ptx::mbar_wait_bounded(full + i, 0);
            ptx::mbar_wait_bounded(full + i, 1);
        }
    }
#pragma unroll
    for (int e = 0; e < 2 * P; ++e) {
        const int j = column(e);
        if (j >= cols) continue;
        float *p = a.part + int64_t(blockIdx.x) * 2 * cols + j;
        if (TR_STORE_OK(sp, p, 4)) *p = e & 1 ? dg[e / 2].y : dg[e / 2].x;
        if (TR_STORE_OK(sp, p + cols, 4)) p[cols] = e & 1 ? db[e / 2].y : db[e / 2].x;
    }
}

// dx of one row per block, in two walks along it: rows that the ring does not hold.
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

// The parts' sums: 32 columns by 8 rows of threads, each over every eighth part,
// joined in a fixed order.
__global__ void __launch_bounds__(256) k_ln_join(Bwd a) {
    pdl_prologue();
    __shared__ float red[8][33];
    [[maybe_unused]] const dbg::Side sp = dbg::side(a.part, 1, 2 * a.parts, a.cols, a.cols, 0, 4);
    [[maybe_unused]] const dbg::Side so = dbg::side(blockIdx.y ? a.dbeta : a.dgamma, 1, 1, a.cols, a.cols, 0, 4);
    float *out = blockIdx.y ? a.dbeta : a.dgamma;
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    for (int64_t c0 = int64_t(blockIdx.x) * 32; c0 < a.cols; c0 += int64_t(gridDim.x) * 32) {
        const int64_t j = c0 + tx;
        float s = 0.0f;
        if (j < a.cols)
#pragma unroll 8
            for (int64_t i = ty; i < a.parts; i += 8) {
                const float *p = a.part + (2 * i + blockIdx.y) * a.cols + j;
                if (TR_LOAD_OK(sp, p, 4)) s += *p;
            }
        red[ty][tx] = s;
        __syncthreads();
        if (ty == 0 && j < a.cols) {
#pragma unroll
            for (int k = 1; k < 8; ++k) s += red[k][tx];
            if (TR_STORE_OK(so, out + j, 4)) out[j] = s;
        }
        __syncthreads();
    }
}

cudaError_t launch_join(const Bwd &a, cudaStream_t stream) {
    const int64_t strips = (a.cols + 31) / 32, most = 1 << 20;
    return launch_pdl(k_ln_join, dim3(unsigned(strips < most ? strips : most), a.dbeta ? 2 : 1), dim3(256), 0, stream, a);
}

// Most blocks that leave sums of their own, from the sizes alone: the more, the
// more bytes to join, the fewer, the fewer rows in flight.
int64_t most_parts(int64_t rows, int64_t cols) {
    const int64_t n = cols <= 1024 ? 1216 : cols <= 2048 ? 608 : 304;
    return rows < n ? rows : n;
}

int64_t parts_of(int64_t rows) {  // of k_ln_columns
    const int64_t n = (rows + 63) / 64;
    return n < 64 ? n : 64;
}

// The ring kernel's launch; cudaErrorNotSupported where a ring of two rows does
// not fit.
template <typename T>
cudaError_t launch_ring(Bwd a, bool vec, cudaStream_t stream) {
    if (a.cols > 16384) return cudaErrorNotSupported;
    const bool keep = a.cols <= 8192;
    int threads = 64;
    while (threads * 16 < a.cols) threads *= 2;
    const uint32_t row_bytes = uint32_t((a.cols * int64_t(sizeof(T)) + 30) / 16 * 16);
    const uint32_t weights = keep ? 0 : uint32_t(a.cols * 4 + 15) / 16 * 16;
    // 512 (1024) threads to an SM, in as many blocks; fewer where rows or the ring want it.
    int64_t per_sm = keep ? 512 / threads : 1;
    const int64_t cap = most_parts(a.rows, a.cols) / sm_count();
    if (per_sm > cap) per_sm = cap < 1 ? 1 : cap;
    uint32_t stages = (ring_room(per_sm) - weights) / (2 * row_bytes);
    while (stages < 4 && per_sm > 1) {
        per_sm /= 2;
        stages = (ring_room(per_sm) - weights) / (2 * row_bytes);
    }
    if (stages < 2) return cudaErrorNotSupported;
    if (stages > kMaxStages) stages = kMaxStages;
    a.parts = int64_t(sm_count()) * per_sm;
    if (a.parts > most_parts(a.rows, a.cols)) a.parts = most_parts(a.rows, a.cols);
    const size_t smem = size_t(stages) * 2 * row_bytes + weights;
    auto run = [&](auto kern) {
        // Always the most that any call needs: threads with rows of other lengths set it too.
        const cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(ring_room(1)));
        if (err != cudaSuccess) return err;
        return launch_pdl(kern, dim3(unsigned(a.parts)), dim3(unsigned(threads)), smem, stream, a, int(stages), row_bytes);
    };
    cudaError_t err;
    if (keep) err = vec ? run(k_ln_backward<T, true, true>) : run(k_ln_backward<T, true, false>);
    else err = vec ? run(k_ln_backward<T, false, true>) : run(k_ln_backward<T, false, false>);
    return err == cudaSuccess ? launch_join(a, stream) : err;
}

template <typename T>
cudaError_t launch_typed(Bwd a, cudaStream_t stream) {
    constexpr int V = 16 / int(sizeof(T));
    const bool vec = a.cols % V == 0 && side_aligned16(a.x, a.ld_x, 0, 1, sizeof(T)) &&
                     side_aligned16(a.dy, a.ld_dy, 0, 1, sizeof(T)) && side_aligned16(a.dx, a.ld_dx, 0, 1, sizeof(T));
    cudaError_t e = launch_ring<T>(a, vec, stream);
    if (e != cudaErrorNotSupported) return e;
    a.parts = parts_of(a.rows);
    a.rows_per_part = (a.rows + a.parts - 1) / a.parts;
    const uintptr_t ax = reinterpret_cast<uintptr_t>(a.x), ad = reinterpret_cast<uintptr_t>(a.dy),
                    ao = reinterpret_cast<uintptr_t>(a.dx);
    const bool alike = (((ax ^ ad) | (ax ^ ao)) & 15u) == 0 &&
                       ((a.ld_x - a.ld_dy) * int64_t(sizeof(T))) % 16 == 0 &&
                       ((a.ld_x - a.ld_dx) * int64_t(sizeof(T))) % 16 == 0;
    const int64_t most = int64_t(1) << 30;
    const dim3 rows_grid(unsigned(a.rows < most ? a.rows : most));
    e = alike ? launch_pdl(k_ln_dx<T, V>, rows_grid, dim3(512), 0, stream, a)
              : launch_pdl(k_ln_dx<T, 1>, rows_grid, dim3(512), 0, stream, a);
    if (e != cudaSuccess) return e;
    const int64_t strips = (a.cols + 31) / 32;
    const dim3 grid(unsigned(strips < most ? strips : most), unsigned(a.parts));
    e = launch_pdl(k_ln_columns<T>, grid, dim3(256), 0, stream, a);
    return e == cudaSuccess ? launch_join(a, stream) : e;
}

__global__ void k_wait_selftest_layernorm(int arrive, uint64_t limit_ns) {
    wait_selftest(&g_fault_flag_layernorm, arrive, limit_ns);
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
    const Bwd a{p.dy, p.x, p.gamma, p.mean, p.rstd, p.dx, p.dgamma, p.dbeta,
          static_cast<float *>(p.workspace), p.rows, p.cols, p.ld_dy, p.ld_x, p.ld_dx,
          0, 0, p.w_dtype == TR_DTYPE_BF16};
    return p.x_dtype == TR_DTYPE_F32 ? launch_typed<float>(a, stream) : launch_typed<__nv_bfloat16>(a, stream);
}

cudaError_t launch_wait_selftest_layernorm(bool arrive, int64_t limit_ns, cudaStream_t stream) {
    k_wait_selftest_layernorm<<<1, 32, 0, stream>>>(arrive ? 1 : 0, uint64_t(limit_ns));
    return cudaGetLastError();
}

cudaError_t read_and_clear_fault_layernorm(unsigned *value) {
    cudaError_t e = cudaMemcpyFromSymbol(value, g_fault_flag_layernorm, sizeof(unsigned));
    if (e != cudaSuccess) return e;
    const unsigned zero = 0;
    return cudaMemcpyToSymbol(g_fault_flag_layernorm, &zero, sizeof(unsigned));
}

}  // namespace tr

extern "C" int64_t tr_layernorm_backward_workspace(int64_t rows, int64_t cols) {
    if (rows < 0 || cols < 0) return -1;
    if (rows == 0 || cols == 0) return 0;
    int64_t n;
    if (!tr::mul_add(cols, 8 * tr::most_parts(rows, cols), 0, &n)) return -1;
    return n;
}

// Root-mean-square norm, backward: the gradient of what was normed along the rows, the
// weight's down the columns.  With u = h * rstd and g = dy * gamma,
//
//   dx = rstd * (g - u * sum(g u)/n) + dresidual,  dgamma = sum_rows dy u
//
// Bound by memory: one read of dy, h and dresidual, one write of dx.  A block walks its rows once, through a ring that
// bulk copies fill, keeps a row's g and u in registers between the row's sum and dx, and holds its columns' part of dgamma
// in registers throughout; a second launch adds the blocks' parts in a fixed order.  Device time, and the share of the
// copy rate: 256 x 1024 bf16 7.0 us; 16384 x 8192 bf16 161 us (98%), 12289 x 7919 fp32 225 (102%), 65536 x 1024 bf16 122
// (65%), 4096 x 16384 bf16 186 (43%).  Rows that the ring does not hold take three launches, and dy and h are read twice:
// 4096 x 16384 fp32 329 us (48%), 4000 x 20000 bf16 224 (42%).
#include "launch.cuh"
#include "ptx.cuh"
#include "row_chunk.cuh"
#include "row_ring.cuh"
#include "tr_internal.h"
#include "wait_selftest.cuh"

namespace tr {

// Set when a bounded in-kernel wait ran out; read and cleared by the host.
__device__ unsigned g_fault_flag_rmsnorm_backward = 0;

namespace {

struct RmsBwd {
    const void *dy, *h, *gamma;
    const float *rstd;
    const void *dres;
    void *dx;
    float *dgamma, *part;
    int64_t rows, cols, ld_dy, ld_h, ld_dres, ld_dx;
    int64_t parts, rows_per_part;
    bool w_bf16, w_held;  // w_held: the ring leaves room for the weights
};

// Sum over the block, in every thread; `slot` holds a word for each of 32 warps.
__device__ __forceinline__ float block_sum(float v, float *slot) {
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    v = warp_sum(v);
    if (lane == 0) slot[threadIdx.x >> 5] = v;
    __syncthreads();
    return warp_sum(lane < warps ? slot[lane] : 0.0f);
}

// The rows' gradients and the columns' sums from one read.  A resident block walks rows; bulk copies keep a
// ring of its next rows of h, dy and dresidual in flight, so no register holds loaded data and any
// alignment reads whole granules.  A thread owns the same 16 columns of every row and sums their dy*u in
// registers (two columns to an instruction); the blocks' sums are joined by k_rms_join.  VEC:
// columns in 16-byte chunks, every row on a 16-byte boundary; else one column at a time, neighbouring
// threads on neighbouring columns.  KEEP (up to 8192 columns): 512 threads to an SM, with a row's u, g and
// dresidual in registers between its two walks; else 1024, which read them from the ring again, and the
// weights from shared memory, or from L2 where the rows leave no room for them (4096 x 16384 bf16 186 us, 588 with
// k_rms_dx and k_rms_columns value by value).
template <typename T, bool KEEP, bool VEC>
__global__ void __launch_bounds__(KEEP ? 512 : 1024, 1)
k_rms_backward(const RmsBwd a, int stages, uint32_t row_bytes) {
    constexpr int V = VEC ? 16 / int(sizeof(T)) : 1;
    constexpr int P = 8;  // pairs of columns to a thread
    extern __shared__ uint4 ring4[];
    __shared__ uint64_t full[kMaxStages];
    __shared__ float slots[2][32];
    const bool add = a.dres != nullptr;
    const uint32_t stage_bytes = (add ? 3 : 2) * row_bytes;
    uint8_t *ring = reinterpret_cast<uint8_t *>(ring4);
    float *gammas = reinterpret_cast<float *>(ring + size_t(stages) * stage_bytes);  // without KEEP
    [[maybe_unused]] const dbg::Side sd = dbg::side(a.dy, 1, a.rows, a.cols, a.ld_dy, 0, sizeof(T));
    [[maybe_unused]] const dbg::Side sh = dbg::side(a.h, 1, a.rows, a.cols, a.ld_h, 0, sizeof(T));
    [[maybe_unused]] const dbg::Side se = dbg::side(a.dres, 1, a.rows, a.cols, a.ld_dres, 0, sizeof(T));
    [[maybe_unused]] const dbg::Side so = dbg::side(a.dx, 1, a.rows, a.cols, a.ld_dx, 0, sizeof(T));
    [[maybe_unused]] const dbg::Side sw = dbg::side(a.gamma, 1, 1, a.cols, a.cols, 0, a.w_bf16 ? 2 : 4);
    [[maybe_unused]] const dbg::Side sr = dbg::side(a.rstd, 1, 1, a.rows, a.rows, 0, 4);
    [[maybe_unused]] const dbg::Side sp = dbg::side(a.part, 1, a.parts, a.cols, a.cols, 0, 4);
    const int t = threadIdx.x, nt = blockDim.x, cols = int(a.cols);
    if (t == 0) {
        for (int i = 0; i < stages; ++i) ptx::mbar_init(full + i, 1);
        ptx::fence_barrier_init();
    }
    __syncthreads();
    pdl_prologue();
    auto granules_of = [&](int64_t row, Granules (&g)[3]) {
        g[0] = granules<T>(a.h, a.rows, a.cols, a.ld_h, row);
        g[1] = granules<T>(a.dy, a.rows, a.cols, a.ld_dy, row);
        g[2] = add ? granules<T>(a.dres, a.rows, a.cols, a.ld_dres, row) : Granules{nullptr, 0, 0, true};
        return g[0].inside && g[1].inside && g[2].inside;
    };
    auto issue = [&](int64_t row, int stage) {  // one thread
        Granules g[3];
        if (!granules_of(row, g)) {  // the block copies that row itself
            ptx::mbar_arrive(full + stage);
            return;
        }
        uint8_t *at = ring + size_t(stage) * stage_bytes;
        ptx::mbar_arrive_expect_tx(full + stage, g[0].bytes + g[1].bytes + g[2].bytes);
        ptx::bulk_load(at, g[0].src, g[0].bytes, full + stage);
        ptx::bulk_load(at + row_bytes, g[1].src, g[1].bytes, full + stage);
        if (add) ptx::bulk_load(at + 2 * row_bytes, g[2].src, g[2].bytes, full + stage);
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
    auto kept = [&](int j) { return j < cols ? weight(a.gamma, a.w_bf16, j, sw) : 0.0f; };
    float2 w[KEEP ? P : 1], dg[P];
#pragma unroll
    for (int k = 0; k < P; ++k) {
        dg[k] = make_float2(0.0f, 0.0f);
        if (KEEP) w[KEEP ? k : 0] = make_float2(kept(column(2 * k)), kept(column(2 * k + 1)));
    }
    if (!KEEP && a.w_held) {
        for (int j = t; j < cols; j += nt) gammas[j] = kept(j);
        __syncthreads();
    }
    auto weights = [&](int k) {
        if (KEEP) return w[KEEP ? k : 0];
        const int j0 = column(2 * k), j1 = column(2 * k + 1);
        if (!a.w_held) return make_float2(kept(j0), kept(j1));
        return make_float2(j0 < cols ? gammas[j0] : 0.0f, j1 < cols ? gammas[j1] : 0.0f);
    };
    const float inv_cols = 1.0f / float(cols);
    auto stat = [&](int64_t row) { return row < a.rows && TR_LOAD_OK(sr, a.rstd + row, 4) ? a.rstd[row] : 0.0f; };
    float rstd_next = stat(blockIdx.x);
    bool ok = true;
    int stage = 0, turn = 0;
    uint32_t phase = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const float rstd = rstd_next;
        rstd_next = stat(row + gridDim.x);
        if (ok) ok = ptx::mbar_wait_bounded(full + stage, phase);
        uint8_t *at = ring + size_t(stage) * stage_bytes;
        T *ph = reinterpret_cast<T *>(at), *pd = reinterpret_cast<T *>(at + row_bytes), *pe = reinterpret_cast<T *>(at + 2 * row_bytes);
        if constexpr (!VEC) {
            Granules g[3];
            const bool inside = granules_of(row, g);
            ph = reinterpret_cast<T *>(at + g[0].shift);
            pd = reinterpret_cast<T *>(at + row_bytes + g[1].shift);
            pe = reinterpret_cast<T *>(at + 2 * row_bytes + g[2].shift);
            if (!inside) {
                const T *hr = static_cast<const T *>(a.h) + row * a.ld_h;
                const T *dr = static_cast<const T *>(a.dy) + row * a.ld_dy;
                const T *er = static_cast<const T *>(a.dres) + row * a.ld_dres;
                for (int j = t; j < cols; j += nt) {
                    if (TR_LOAD_OK(sh, hr + j, int(sizeof(T)))) ph[j] = hr[j];
                    if (TR_LOAD_OK(sd, dr + j, int(sizeof(T)))) pd[j] = dr[j];
                    if (add && TR_LOAD_OK(se, er + j, int(sizeof(T)))) pe[j] = er[j];
                }
                ptx::fence_proxy_async_smem();
                __syncthreads();
            }
        }
        const float2 rstd2 = make_float2(rstd, rstd);
        float2 u[KEEP ? P : 1], g[KEEP ? P : 1], e[KEEP ? P : 1], s2 = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < P / Q; ++i) {
            float2 h2[Q], d2[Q], e2[Q];
            piece(ph, i, h2);
            piece(pd, i, d2);
            if (KEEP && add) piece(pe, i, e2);
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                const int k = i * Q + q;
                const float2 uk = __fmul2_rn(h2[q], rstd2), gk = __fmul2_rn(d2[q], weights(k));
                dg[k] = __ffma2_rn(d2[q], uk, dg[k]);
                s2 = __ffma2_rn(gk, uk, s2);
                if (KEEP) {
                    u[KEEP ? k : 0] = uk;
                    g[KEEP ? k : 0] = gk;
                    e[KEEP ? k : 0] = add ? e2[q] : make_float2(0.0f, 0.0f);
                }
            }
        }
        const float s = block_sum(s2.x + s2.y, slots[turn]);
        // Past its meeting the block has read this row (KEEP), or left the last one.
        if (t == 0 && ok && (KEEP || row != blockIdx.x)) {
            const int64_t next = row + int64_t(KEEP ? stages : stages - 1) * gridDim.x;
            if (next < a.rows) issue(next, KEEP ? stage : stage == 0 ? stages - 1 : stage - 1);
        }
        const float2 minus_c = make_float2(-s * inv_cols, -s * inv_cols);
        T *out = static_cast<T *>(a.dx) + row * a.ld_dx;
#pragma unroll
        for (int i = 0; i < P / Q; ++i) {
            float2 h2[Q], d2[Q], e2[Q];
            if (!KEEP) {
                piece(ph, i, h2);
                piece(pd, i, d2);
                if (add) piece(pe, i, e2);
            }
            float v[2 * Q];
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                const int k = i * Q + q;
                const float2 uk = KEEP ? u[KEEP ? k : 0] : __fmul2_rn(h2[q], rstd2);
                const float2 gk = KEEP ? g[KEEP ? k : 0] : __fmul2_rn(d2[q], weights(k));
                const float2 ek = KEEP ? e[KEEP ? k : 0] : add ? e2[q] : make_float2(0.0f, 0.0f);
                const float2 r = __ffma2_rn(rstd2, __ffma2_rn(uk, minus_c, gk), ek);
                v[2 * q] = r.x;
                v[2 * q + 1] = r.y;
            }
            constexpr int PIECES = 2 * Q / V;  // that are stored
#pragma unroll
            for (int m = 0; m < PIECES; ++m) {
                const int j = column((i * PIECES + m) * V);
                if (j >= cols) continue;
                Pack<T, V> o;
                float whole[V];
#pragma unroll
                for (int q = 0; q < V; ++q) whole[q] = v[m * V + q];
                o.round(whole);
                store_chunk<T, V, false>(out, j, cols, o, so);
            }
        }
        turn ^= 1;
        if (++stage == stages) {
            stage = 0;
            phase ^= 1;
        }
    }
    if (!ok) {
        atomicExch(&g_fault_flag_rmsnorm_backward, 1u);
        for (int i = 0; i < stages; ++i) {  // no copy may land after the block has gone
            ptx::mbar_wait_bounded(full + i, 0);
            ptx::mbar_wait_bounded(full + i, 1);
        }
    }
#pragma unroll
    for (int e = 0; e < 2 * P; ++e) {
        const int j = column(e);
        if (j >= cols) continue;
        float *p = a.part + int64_t(blockIdx.x) * cols + j;
        if (TR_STORE_OK(sp, p, 4)) *p = e & 1 ? dg[e / 2].y : dg[e / 2].x;
    }
}

// dx of one row per block, in two walks along it: rows that the ring does not hold.  V: values to an access, rows and
// weights on 16-byte boundaries with more than one (4096 x 16384 fp32 329 us, value by value 570).
template <typename T, int V>
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
        // g and u of the V columns from j on.
        auto values = [&](int64_t j, float (&g)[V], float (&u)[V]) {
            const Pack<T, V> pd = load_chunk<T, V, false>(dy, j, a.cols, sd), ph = load_chunk<T, V, false>(h, j, a.cols, sh);
            if constexpr (V > 1) load_weights<V>(a.gamma, a.w_bf16, j, g, sw);
            else g[0] = weight(a.gamma, a.w_bf16, j, sw);
#pragma unroll
            for (int q = 0; q < V; ++q) {
                g[q] = pd.get(q) * g[q];
                u[q] = ph.get(q) * rstd;
            }
        };
        float s[1] = {0.0f};
#pragma unroll 2
        for (int64_t j = int64_t(threadIdx.x) * V; j < a.cols; j += int64_t(blockDim.x) * V) {
            float g[V], u[V];
            values(j, g, u);
#pragma unroll
            for (int q = 0; q < V; ++q) s[0] = fmaf(g[q], u[q], s[0]);
        }
        group_sum<512, 1>(s, slots[turn]);
        const float c = s[0] * inv_cols;
#pragma unroll 2
        for (int64_t j = int64_t(threadIdx.x) * V; j < a.cols; j += int64_t(blockDim.x) * V) {
            float g[V], u[V];
            values(j, g, u);
            Pack<T, V> pe;
            pe.clear();
            if (a.dres) pe = load_chunk<T, V, false>(dr, j, a.cols, se);
#pragma unroll
            for (int q = 0; q < V; ++q) g[q] = fmaf(rstd, fmaf(-u[q], c, g[q]), pe.get(q));
            Pack<T, V> o;
            o.round(g);
            store_chunk<T, V, false>(dx, j, a.cols, o, so);
        }
    }
}

// Column sums of dy*u over one part of the rows: 32 times V columns by 8 rows of threads.
template <typename T, int V>
__global__ void __launch_bounds__(256) k_rms_columns(const RmsBwd a) {
    pdl_prologue();
    __shared__ float red[8][32 * V + 1];
    [[maybe_unused]] const dbg::Side sd = dbg::side(a.dy, 1, a.rows, a.cols, a.ld_dy, 0, sizeof(T));
    [[maybe_unused]] const dbg::Side sh = dbg::side(a.h, 1, a.rows, a.cols, a.ld_h, 0, sizeof(T));
    [[maybe_unused]] const dbg::Side sp = dbg::side(a.part, 1, a.parts, a.cols, a.cols, 0, 4);
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int64_t part = blockIdx.y;
    const int64_t r0 = part * a.rows_per_part;
    const int64_t r1 = r0 + a.rows_per_part < a.rows ? r0 + a.rows_per_part : a.rows;
    for (int64_t c0 = int64_t(blockIdx.x) * 32 * V; c0 < a.cols; c0 += int64_t(gridDim.x) * 32 * V) {
        const int64_t j = c0 + tx * V;
        float s[V] = {};
        if (j < a.cols)
#pragma unroll 2
            for (int64_t r = r0 + ty; r < r1; r += 8) {
                const Pack<T, V> pd = load_chunk<T, V, false>(static_cast<const T *>(a.dy) + r * a.ld_dy, j, a.cols, sd);
                const Pack<T, V> ph = load_chunk<T, V, false>(static_cast<const T *>(a.h) + r * a.ld_h, j, a.cols, sh);
                const float rstd = a.rstd[r];
#pragma unroll
                for (int q = 0; q < V; ++q) s[q] = fmaf(pd.get(q), ph.get(q) * rstd, s[q]);
            }
#pragma unroll
        for (int q = 0; q < V; ++q) red[ty][tx * V + q] = s[q];
        __syncthreads();
        for (int c = threadIdx.x; c < 32 * V; c += 256)
            if (c0 + c < a.cols) {
                float sum = red[0][c];
#pragma unroll
                for (int i = 1; i < 8; ++i) sum += red[i][c];
                float *p = a.part + part * a.cols + c0 + c;
                if (TR_STORE_OK(sp, p, 4)) *p = sum;
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

cudaError_t launch_join(const RmsBwd &a, cudaStream_t stream) {
    const int64_t strips = (a.cols + 31) / 32, most = 1 << 20;
    return launch_pdl(k_rms_join, dim3(unsigned(strips < most ? strips : most)), dim3(256), 0, stream, a);
}

// The ring kernel's launch; cudaErrorNotSupported where a ring of two rows does not fit.
template <typename T>
cudaError_t launch_ring(RmsBwd a, bool vec, cudaStream_t stream) {
    if (a.cols > 16384) return cudaErrorNotSupported;
    const bool keep = a.cols <= 8192;
    int threads = 64;
    while (threads * 16 < a.cols) threads *= 2;
    const uint32_t row_bytes = uint32_t((a.cols * int64_t(sizeof(T)) + 30) / 16 * 16), stage_bytes = (a.dres ? 3 : 2) * row_bytes;
    uint32_t weights = keep ? 0 : uint32_t(a.cols * 4 + 15) / 16 * 16;
    if (ring_room(1) < weights + 2 * stage_bytes) weights = 0;  // one block to an SM
    a.w_held = weights != 0;
    // 512 (1024) threads to an SM, in as many blocks; fewer where rows or the ring want it.
    int64_t per_sm = keep ? 512 / threads : 1;
    const int64_t cap = most_parts(a.rows, a.cols) / sm_count();
    if (per_sm > cap) per_sm = cap < 1 ? 1 : cap;
    uint32_t stages = (ring_room(per_sm) - weights) / stage_bytes;
    while (stages < 4 && per_sm > 1) {
        per_sm /= 2;
        stages = (ring_room(per_sm) - weights) / stage_bytes;
    }
    if (stages < 2) return cudaErrorNotSupported;
    if (stages > kMaxStages) stages = kMaxStages;
    a.parts = int64_t(sm_count()) * per_sm;
    if (a.parts > most_parts(a.rows, a.cols)) a.parts = most_parts(a.rows, a.cols);
    const size_t smem = size_t(stages) * stage_bytes + weights;
    auto run = [&](auto allowed, auto kern) {
        if (allowed != cudaSuccess) return allowed;
        return launch_pdl(kern, dim3(unsigned(a.parts)), dim3(unsigned(threads)), smem, stream, a, int(stages), row_bytes);
    };
#define TR_RING(KEEP, VEC)  /* always the most shared memory that any call needs */ \
    run(allow_shared<k_rms_backward<T, KEEP, VEC>>(ring_room(1)), k_rms_backward<T, KEEP, VEC>)
    const cudaError_t err = keep ? (vec ? TR_RING(true, true) : TR_RING(true, false)) : (vec ? TR_RING(false, true) : TR_RING(false, false));
#undef TR_RING
    return err == cudaSuccess ? launch_join(a, stream) : err;
}

template <typename T>
cudaError_t launch_typed(RmsBwd a, cudaStream_t stream) {
    constexpr int es = int(sizeof(T));
    const bool vec = a.cols % (16 / es) == 0 && side_aligned16(a.h, a.ld_h, 0, 1, es) && side_aligned16(a.dy, a.ld_dy, 0, 1, es) &&
                     side_aligned16(a.dx, a.ld_dx, 0, 1, es) && (!a.dres || side_aligned16(a.dres, a.ld_dres, 0, 1, es));
    cudaError_t e = launch_ring<T>(a, vec, stream);
    if (e != cudaErrorNotSupported) return e;
    a.parts = parts_of(a.rows);
    a.rows_per_part = (a.rows + a.parts - 1) / a.parts;
    const int64_t most = int64_t(1) << 30;
    auto run = [&](auto dx, auto columns, int64_t strip) {
        const cudaError_t err = launch_pdl(dx, dim3(unsigned(a.rows < most ? a.rows : most)), dim3(512), 0, stream, a);
        const int64_t strips = (a.cols + strip - 1) / strip;
        return err != cudaSuccess ? err : launch_pdl(columns, dim3(unsigned(strips < most ? strips : most), unsigned(a.parts)), dim3(256), 0, stream, a);
    };
    e = vec && (reinterpret_cast<uintptr_t>(a.gamma) & 15u) == 0 ? run(k_rms_dx<T, 16 / es>, k_rms_columns<T, 16 / es>, 32 * 16 / es)
                                                                : run(k_rms_dx<T, 1>, k_rms_columns<T, 1>, 32);
    return e == cudaSuccess ? launch_join(a, stream) : e;
}

}  // namespace

TR_WAIT_UNIT(rmsnorm_backward)

// Debug builds: this unit's record of refused accesses.
TR_BOUNDS_READER(read_bounds_rmsnorm_backward)

cudaError_t launch_rmsnorm_backward(const tr_rmsnorm_backward_args &p) {
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(p.stream);
    if (p.rows == 0) return cudaMemsetAsync(p.dgamma, 0, size_t(p.cols) * 4, stream);  // the column sums are empty
    const RmsBwd a{p.dy, p.h, p.gamma, p.rstd, p.dresidual, p.dx, p.dgamma, static_cast<float *>(p.workspace),
                   p.rows, p.cols, p.ld_dy, p.ld_h, p.ld_dresidual, p.ld_dx, 0, 0, p.w_dtype == TR_DTYPE_BF16, true};
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

// Quantizing to 8-bit floating point with a scale for each block of 128, row
// by row and transposed from one read.  For a block with largest magnitude m and T the
// type's largest value: a = max(m, 2^-100), scale = a / T, q = round(x * (T / a)).
//
// Bound by memory: x is read once and each wanted operand written once, 2 + 1 + 1
// bytes to a bf16 value both ways.  Two things keep it there: a tile is read into
// registers once for both directions, and the work on a value is cut to about eight
// instructions (magnitudes in packed pairs, one division to a row and to a column, two
// values to a conversion).  With the magnitudes in fp32, a division in each
// thread and every thread reading eight warps' column maxima, 16384 x 8192 bf16
// both ways took 277 us.
//
// Measured on one GB300 (share of the measured copy rate, 6771 GB/s):
//   16384 x 8192 bf16, 1 x 128 blocks, both ways   95 us, 5.7 TB/s (85%); rows alone 64 us (92%)
//   16384 x 8192 bf16, 128 x 128, both ways        87 us, 6.2 TB/s (91%)
//   12289 x 7919 fp32, 128 x 128, both ways       124 us, 4.7 TB/s (70%)  (rows off 16-byte boundaries)
//   12288 x 7920 fp32, 128 x 128, both ways       101 us, 5.8 TB/s (85%)
//   12289 x 7919 bf16, 1 x 128, both ways          87 us, 4.5 TB/s (66%)  (rows off 16-byte boundaries)
// Rows off boundaries go through shared memory, and a block waits for all of a tile's
// copies before it works on any: nothing of the next tile is in flight meanwhile.
//   1 x 8192 bf16                                 2.6 us: a launch
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <atomic>

#include "bounds.cuh"
#include "granule.cuh"
#include "launch.cuh"
#include "ptx.cuh"
#include "tr_internal.h"

namespace tr {
namespace {

constexpr int kThreads = 256;
constexpr uint32_t kFloorBits = 0x0D800000u;  // 2^-100

struct Quant {
    const void *x;
    uint8_t *q, *qt;
    float *scale, *scale_t;
    int64_t rows, cols, ld_x, ld_q, ld_scale, ld_qt, ld_scale_t;
    int64_t tiles_r, tiles_c;
    float top;  // the 8-bit type's largest finite value
};

// Eight values times r as eight bytes, the first lowest.
template <bool E5M2>
__device__ __forceinline__ uint2 to_bytes(const float (&v)[8], float r) {
    constexpr __nv_fp8_interpretation_t K = E5M2 ? __NV_E5M2 : __NV_E4M3;
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = __nv_cvt_float2_to_fp8x2(make_float2(v[2 * i] * r, v[2 * i + 1] * r), __NV_SATFINITE, K);
    return make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
}

// Eight bytes of one row at column c (a multiple of 8), those below `cols` only.
__device__ __forceinline__ void store8(uint8_t *row, int64_t c, int64_t cols, uint2 v,
                                       const dbg::Side &s) {
    if (c + 8 <= cols) {
        if (TR_STORE_OK(s, row + c, 8)) *reinterpret_cast<uint2 *>(row + c) = v;
        return;
    }
    for (int i = 0; i < 8 && c + i < cols; ++i)
        if (TR_STORE_OK(s, row + c + i, 1)) row[c + i] = uint8_t((i < 4 ? v.x >> (8 * i) : v.y >> (8 * (i - 4))));
}

// How a tile's values reach the registers.  The two for rows off 16-byte boundaries go
// through shared memory; each warp copies, and reads back, its own 16 rows.
enum Load {
    kVector,   // 16-byte loads: base and pitch on 16-byte boundaries
    kWords,    // fp32: 4-byte asynchronous copies, coalesced (12289 x 7919, 128 x 128 blocks, both
               // ways: 125 us; 16-byte copies of the granules around a row: 152)
    kGranules  // bf16: 16-byte asynchronous copies of the granules around a row, shifted in
               // registers (12289 x 7919, both ways: 86 us; one element at a time: 118)
};

constexpr int kWordPitch = 132;    // fp32 words to a row of the shared tile: rows stay 16-byte aligned
constexpr int kGranulePitch = 72;  // words to a row of 17 granules
constexpr size_t kTileBytes[3] = {0, size_t(128) * kWordPitch * 4, size_t(128) * kGranulePitch * 4};

// One granule of a bf16 row of `cols` values from `row` on, the one that begins at column
// col: its bytes inside the row are copied, those past its end zeroed, and those
// before its start left as they are (nobody reads them).
__device__ __forceinline__ void copy_granule(uint32_t *dst, const __nv_bfloat16 *row, int64_t col, int64_t cols,
                                             const dbg::Side &s) {
    if (col >= 0) {
        const GranulePart p = granule_part(row, col, cols);
        if (p.src && TR_LOAD_OK(s, p.src, p.bytes)) ptx::cp_async_16_or_zero(dst, p.src, p.bytes);
        else *reinterpret_cast<uint4 *>(dst) = make_uint4(0u, 0u, 0u, 0u);
    } else {
        __nv_bfloat16 *e = reinterpret_cast<__nv_bfloat16 *>(dst);
#pragma unroll
        for (int q = 0; q < 8; ++q)
            if (col + q >= 0) e[q] = col + q < cols && TR_LOAD_OK(s, row + col + q, 2) ? row[col + q] : __nv_bfloat16(0.0f);
    }
}

// The 16 bytes from `shift` (even, below 16) on of two granules: whole words move in two
// selections, half a word in a third.
__device__ __forceinline__ uint4 pick(const uint32_t *granules, uint32_t shift) {
    const uint4 a = *reinterpret_cast<const uint4 *>(granules), b = *reinterpret_cast<const uint4 *>(granules + 4);
    uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int k = 0; k < 6; ++k) w[k] = shift & 8 ? w[k + 2] : w[k];
#pragma unroll
    for (int k = 0; k < 5; ++k) w[k] = shift & 4 ? w[k + 1] : w[k];
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = shift & 2 ? __byte_perm(w[k], w[k + 1], 0x5432) : w[k];
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// The 8 x 8 values of one thread.  bf16 stays packed in pairs along the row.
template <typename T>
struct Values;
template <>
struct Values<__nv_bfloat16> {
    uint32_t w[8][4];
    __device__ __forceinline__ float at(int i, int j) const {
        return __uint_as_float(j & 1 ? w[i][j >> 1] & 0xffff0000u : w[i][j >> 1] << 16);
    }
    __device__ __forceinline__ void row(int i, const uint4 *v) {
        w[i][0] = v[0].x;
        w[i][1] = v[0].y;
        w[i][2] = v[0].z;
        w[i][3] = v[0].w;
    }
    __device__ __forceinline__ void set(int i, int j, __nv_bfloat16 v) {
        const uint32_t b = __bfloat16_as_ushort(v);
        w[i][j >> 1] = j & 1 ? (w[i][j >> 1] & 0xffffu) | b << 16 : (w[i][j >> 1] & 0xffff0000u) | b;
    }
};
template <>
struct Values<float> {
    float v[8][8];
    __device__ __forceinline__ float at(int i, int j) const { return v[i][j]; }
    __device__ __forceinline__ void row(int i, const uint4 *r) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            v[i][4 * k] = __uint_as_float(r[k].x);
            v[i][4 * k + 1] = __uint_as_float(r[k].y);
            v[i][4 * k + 2] = __uint_as_float(r[k].z);
            v[i][4 * k + 3] = __uint_as_float(r[k].w);
        }
    }
    __device__ __forceinline__ void set(int i, int j, float x) { v[i][j] = x; }
};

// Larger of two pairs of magnitudes; a NaN wins.
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    const __nv_bfloat162 m = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162 *>(&a),
                                         *reinterpret_cast<const __nv_bfloat162 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&m);
}

__device__ __forceinline__ uint32_t shfl(uint32_t v, int mask) {
    return __shfl_xor_sync(0xffffffffu, v, mask);
}

// Magnitudes of one thread's rows and columns, and the joins over the 16 lanes
// of a row and the two row groups of a warp.  A magnitude is the bits of its
// fp32 value (a NaN is larger than every number there too).
template <typename T>
struct Magnitudes;

template <>
struct Magnitudes<__nv_bfloat16> {
    uint32_t r[4], c[4];  // pairs: rows 2k, 2k+1 and columns 2k, 2k+1
    __device__ __forceinline__ void of(const Values<__nv_bfloat16> &x) {
        uint32_t rows[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t a = x.w[i][k] & 0x7fff7fffu;
                rows[i] = k ? max2(rows[i], a) : a;
                c[k] = i ? max2(c[k], a) : a;
            }
#pragma unroll
        for (int k = 0; k < 4; ++k)
            r[k] = max2(__byte_perm(rows[2 * k], rows[2 * k + 1], 0x5410),
                        __byte_perm(rows[2 * k], rows[2 * k + 1], 0x7632));
    }
    __device__ __forceinline__ uint32_t all() const {
        const uint32_t m = max2(max2(r[0], r[1]), max2(r[2], r[3]));
        return max(m << 16, m & 0xffff0000u);
    }
    // Over the 16 lanes of a row group: lane l ends up with row
    // 4*(l>>3 & 1) + 2*(l>>2 & 1) + (l & 1).
    __device__ __forceinline__ uint32_t row(int lane) const {
        uint32_t a = lane & 8 ? r[2] : r[0], b = lane & 8 ? r[3] : r[1];
        a = max2(a, shfl(lane & 8 ? r[0] : r[2], 8));
        b = max2(b, shfl(lane & 8 ? r[1] : r[3], 8));
        uint32_t m = max2(lane & 4 ? b : a, shfl(lane & 4 ? a : b, 4));
        m = max2(m, shfl(m, 2));
        m = max2(m, shfl(m, 1));
        return lane & 1 ? m & 0xffff0000u : m << 16;
    }
    // Over the warp's two row groups, into eight columns' worth of shared words.
    static constexpr int kBytes = 2;
    __device__ __forceinline__ void columns(int lane, uint8_t *warp_row) const {
        uint4 m;
        m.x = max2(c[0], shfl(c[0], 16));
        m.y = max2(c[1], shfl(c[1], 16));
        m.z = max2(c[2], shfl(c[2], 16));
        m.w = max2(c[3], shfl(c[3], 16));
        if (lane < 16) *reinterpret_cast<uint4 *>(warp_row + lane * 16) = m;
    }
    static __device__ __forceinline__ uint32_t word(const uint8_t *p) {
        return uint32_t(*reinterpret_cast<const uint16_t *>(p)) << 16;
    }
};

template <>
struct Magnitudes<float> {
    uint32_t r[8], c[8];
    __device__ __forceinline__ void of(const Values<float> &x) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const uint32_t a = __float_as_uint(x.v[i][k]) & 0x7fffffffu;
                r[i] = k ? max(r[i], a) : a;
                c[k] = i ? max(c[k], a) : a;
            }
    }
    __device__ __forceinline__ uint32_t all() const {
        uint32_t m = r[0];
#pragma unroll
        for (int i = 1; i < 8; ++i) m = max(m, r[i]);
        return m;
    }
    __device__ __forceinline__ uint32_t row(int lane) const {
        uint32_t a[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = max(lane & 8 ? r[i + 4] : r[i], shfl(lane & 8 ? r[i] : r[i + 4], 8));
        const uint32_t b0 = max(lane & 4 ? a[2] : a[0], shfl(lane & 4 ? a[0] : a[2], 4));
        const uint32_t b1 = max(lane & 4 ? a[3] : a[1], shfl(lane & 4 ? a[1] : a[3], 4));
        uint32_t m = max(lane & 1 ? b1 : b0, shfl(lane & 1 ? b0 : b1, 1));
        return max(m, shfl(m, 2));
    }
    static constexpr int kBytes = 4;
    __device__ __forceinline__ void columns(int lane, uint8_t *warp_row) const {
        uint32_t m[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) m[k] = max(c[k], shfl(c[k], 16));
        if (lane < 16) {
            uint4 *p = reinterpret_cast<uint4 *>(warp_row + lane * 32);
            p[0] = make_uint4(m[0], m[1], m[2], m[3]);
            p[1] = make_uint4(m[4], m[5], m[6], m[7]);
        }
    }
    static __device__ __forceinline__ uint32_t word(const uint8_t *p) {
        return *reinterpret_cast<const uint32_t *>(p);
    }
};

// One 128 x 128 tile per turn.  A thread holds the 8 x 8 values of row group rg
// and column group cg; 16 lanes share a row group, so a row's magnitude is a
// butterfly of shuffles that leaves one row to each lane, and a column's goes
// through shared memory to one thread per column: each T / a and a / T is
// divided once.  Row bytes are stored straight from the registers (16 lanes
// write 128 contiguous bytes); the transposed ones go through a shared tile of
// 8-byte slots, slot XOR column group, so that neither its writes nor its
// reads share a bank.
template <typename T, Load LOAD, bool E5M2, bool BLOCK, bool BOTH>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 4 : 2) k_quantize(const Quant a) {
    pdl_prologue();
    using M = Magnitudes<T>;
    extern __shared__ uint4 shared_tile[];
    __shared__ alignas(16) uint8_t col_max[8][128 * M::kBytes];
    __shared__ alignas(16) float col_inv[128];
    __shared__ uint2 turned[BOTH ? 128 * 16 : 1];
    [[maybe_unused]] const dbg::Side sx = dbg::side(a.x, 1, a.rows, a.cols, a.ld_x, 0, sizeof(T));
    [[maybe_unused]] const dbg::Side sq = dbg::side(a.q, 1, a.rows, a.cols, a.ld_q, 0, 1);
    [[maybe_unused]] const dbg::Side st = dbg::side(a.qt, 1, a.cols, a.rows, a.ld_qt, 0, 1);
    [[maybe_unused]] const dbg::Side ss = dbg::side(a.scale, 1, a.tiles_c, BLOCK ? a.tiles_r : a.rows, a.ld_scale, 0, 4);
    [[maybe_unused]] const dbg::Side su = dbg::side(a.scale_t, 1, a.tiles_r, BLOCK ? a.tiles_c : a.cols, a.ld_scale_t, 0, 4);
    const int t = threadIdx.x, lane = t & 31, cg = t & 15, rg = t >> 4, warp = t >> 5;
    const T *x = static_cast<const T *>(a.x);
    for (int64_t tile = blockIdx.x; tile < a.tiles_r * a.tiles_c; tile += gridDim.x) {
        const int64_t tr = tile / a.tiles_c, tc = tile - tr * a.tiles_c;
        const int64_t r0 = tr * 128 + rg * 8, c0 = tc * 128 + cg * 8;
        Values<T> v;
        if constexpr (LOAD == kWords) {
            float *words = reinterpret_cast<float *>(shared_tile);
#pragma unroll 8
            for (int k = 0; k < 64; ++k) {  // a warp copies 16 rows, 32 columns at a time
                const int r = warp * 16 + (k >> 2), c = (k & 3) * 32 + lane;
                const int64_t row = tr * 128 + r, col = tc * 128 + c;
                float *dst = words + r * kWordPitch + c;
                const T *p = x + row * a.ld_x + col;
                const bool have = row < a.rows && col < a.cols && TR_LOAD_OK(sx, p, 4);
                ptx::cp_async_4_or_zero(dst, have ? p : x, have);
            }
            ptx::cp_async_wait_all();
            __syncwarp();  // a warp reads back only what it copied: rows 16*warp ..
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v.row(i, reinterpret_cast<const uint4 *>(words + (rg * 8 + i) * kWordPitch + cg * 8));
        } else if constexpr (LOAD == kGranules) {
            uint32_t *granules = reinterpret_cast<uint32_t *>(shared_tile) + warp * 16 * kGranulePitch;
            const T *first = x + (tr * 128 + warp * 16) * a.ld_x;  // the warp's first row
            auto shift = [&](int r) { return granule_shift(first + r * a.ld_x + tc * 128); };
            auto copy = [&](int r, int granule) {
                uint32_t *dst = granules + r * kGranulePitch + granule * 4;
                if (tr * 128 + warp * 16 + r < a.rows)
                    copy_granule(dst, first + r * a.ld_x, tc * 128 + granule * 8 - int(shift(r) / 2), a.cols, sx);
                else
                    *reinterpret_cast<uint4 *>(dst) = make_uint4(0u, 0u, 0u, 0u);
            };
            if (tc > 0 && (tc + 1) * 128 + 8 <= a.cols && tr * 128 + 128 <= a.rows) {
                // Inside the matrix every granule is whole: two rows to an instruction,
                // then the last granule of each row.
                auto whole = [&](int r, int granule) {
                    const T *src = first + r * a.ld_x + tc * 128 - shift(r) / 2 + granule * 8;
                    if (TR_LOAD_OK(sx, src, 16)) ptx::cp_async_16(granules + r * kGranulePitch + granule * 4, src);
                };
#pragma unroll
                for (int r = 0; r < 16; r += 2) whole(r + (lane >> 4), lane & 15);
                if (lane < 16) whole(lane, 16);
            } else {
#pragma unroll 1
                for (int k = lane; k < 16 * 17; k += 32) copy(k / 17, k % 17);
            }
            ptx::cp_async_wait_all();
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int r = (rg & 1) * 8 + i;
                const uint4 raw[1] = {pick(granules + r * kGranulePitch + cg * 4, shift(r))};
                v.row(i, raw);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const T *p = x + (r0 + i) * a.ld_x + c0;
                uint4 raw[sizeof(T) / 2] = {};
                if (r0 + i < a.rows && c0 + 8 <= a.cols && TR_LOAD_OK(sx, p, int(8 * sizeof(T)))) {
#pragma unroll
                    for (int k = 0; k < int(sizeof(T)) / 2; ++k) raw[k] = __ldcs(reinterpret_cast<const uint4 *>(p) + k);
                    v.row(i, raw);
                } else {
                    v.row(i, raw);
                    if (r0 + i < a.rows)
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (c0 + j < a.cols && TR_LOAD_OK(sx, p + j, int(sizeof(T)))) v.set(i, j, p[j]);
                }
            }
        }
        M m;
        m.of(v);
        float inv[8];  // T / a of the rows, then of the columns
        if constexpr (BLOCK) {
            uint32_t w = __reduce_max_sync(0xffffffffu, m.all());
            uint32_t *shared = reinterpret_cast<uint32_t *>(col_inv);
            if (lane == 0) shared[warp] = w;
            __syncthreads();
#pragma unroll
            for (int k = 0; k < 8; ++k) w = max(w, shared[k]);
            const float amax = __uint_as_float(max(w, kFloorBits));
            const float one = a.top / amax;
#pragma unroll
            for (int i = 0; i < 8; ++i) inv[i] = one;
            if (t == 0) {
                float *s = a.scale + tc * a.ld_scale + tr;
                if (TR_STORE_OK(ss, s, 4)) *s = amax / a.top;
                if (BOTH) {
                    float *u = a.scale_t + tr * a.ld_scale_t + tc;
                    if (TR_STORE_OK(su, u, 4)) *u = amax / a.top;
                }
            }
        } else {
            if constexpr (BOTH) m.columns(lane, col_max[warp]);
            const float amax = __uint_as_float(max(m.row(lane), kFloorBits));
            const float mine = a.top / amax;
            const int64_t row = r0 + (lane >> 3 & 1) * 4 + (lane >> 2 & 1) * 2 + (lane & 1);
            if ((lane & 2) == 0 && row < a.rows) {
                float *s = a.scale + tc * a.ld_scale + row;
                if (TR_STORE_OK(ss, s, 4)) *s = amax / a.top;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
                inv[i] = __shfl_sync(0xffffffffu, mine, (lane & 16) | (i >> 2) << 3 | (i >> 1 & 1) << 2 | (i & 1));
            if constexpr (BOTH) {
                __syncthreads();
                if (t < 128) {
                    uint32_t w = kFloorBits;
#pragma unroll
                    for (int k = 0; k < 8; ++k) w = max(w, M::word(col_max[k] + t * M::kBytes));
                    const float cmax = __uint_as_float(w);
                    col_inv[t] = a.top / cmax;
                    if (tc * 128 + t < a.cols) {
                        float *u = a.scale_t + tr * a.ld_scale_t + tc * 128 + t;
                        if (TR_STORE_OK(su, u, 4)) *u = cmax / a.top;
                    }
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float row[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) row[j] = v.at(i, j);
            if (r0 + i < a.rows) store8(a.q + (r0 + i) * a.ld_q, c0, a.cols, to_bytes<E5M2>(row, inv[i]), sq);
        }
        if constexpr (BOTH) {
            if constexpr (!BLOCK) {
                __syncthreads();
#pragma unroll
                for (int j = 0; j < 8; j += 4) {
                    const float4 f = *reinterpret_cast<const float4 *>(col_inv + cg * 8 + j);
                    inv[j] = f.x;
                    inv[j + 1] = f.y;
                    inv[j + 2] = f.z;
                    inv[j + 3] = f.w;
                }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float col[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) col[i] = v.at(i, j);
                turned[(cg * 8 + j) * 16 + (rg ^ cg)] = to_bytes<E5M2>(col, inv[j]);
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int c = i * 16 + rg;
                const int64_t col = tc * 128 + c;
                if (col < a.cols)
                    store8(a.qt + col * a.ld_qt, tr * 128 + cg * 8, a.rows, turned[c * 16 + (cg ^ (c >> 3))], st);
            }
        }
        // The shared words are written anew in the next turn.
        if (tile + gridDim.x < a.tiles_r * a.tiles_c) __syncthreads();
    }
}

template <typename T, Load LOAD, bool E5M2, bool BLOCK, bool BOTH>
cudaError_t launch_one(const Quant &a, cudaStream_t stream) {
    auto kern = k_quantize<T, LOAD, E5M2, BLOCK, BOTH>;
    constexpr size_t smem = kTileBytes[LOAD];
    if (smem) {
        static std::atomic<bool> opted[64];  // per device, zero-initialised (static)
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
        if (!opted[dev].load(std::memory_order_acquire)) {  // setting it twice is harmless
            e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
            if (e != cudaSuccess) return e;
            opted[dev].store(true, std::memory_order_release);
        }
    }
    const int64_t tiles = a.tiles_r * a.tiles_c, most = int64_t(1) << 30;
    return launch_pdl(kern, dim3(unsigned(tiles < most ? tiles : most)), dim3(kThreads), smem, stream, a);
}

template <typename T, Load LOAD, bool E5M2>
cudaError_t launch_typed(const Quant &a, bool block, cudaStream_t stream) {
    if (block)
        return a.qt ? launch_one<T, LOAD, E5M2, true, true>(a, stream) : launch_one<T, LOAD, E5M2, true, false>(a, stream);
    return a.qt ? launch_one<T, LOAD, E5M2, false, true>(a, stream) : launch_one<T, LOAD, E5M2, false, false>(a, stream);
}

template <typename T>
cudaError_t launch_in(const Quant &a, bool block, bool e5m2, cudaStream_t stream) {
    constexpr Load kOther = sizeof(T) == 4 ? kWords : kGranules;
    if (side_aligned16(a.x, a.ld_x, 0, 1, sizeof(T)))
        return e5m2 ? launch_typed<T, kVector, true>(a, block, stream) : launch_typed<T, kVector, false>(a, block, stream);
    return e5m2 ? launch_typed<T, kOther, true>(a, block, stream) : launch_typed<T, kOther, false>(a, block, stream);
}

}  // namespace

// Debug builds: this unit's record of refused accesses.
TR_BOUNDS_READER(read_bounds_quantize)

cudaError_t launch_quantize(const tr_quantize_args &p) {
    const bool e5m2 = p.q_dtype == TR_DTYPE_E5M2;
    const Quant a{p.x, static_cast<uint8_t *>(p.q), static_cast<uint8_t *>(p.qt), p.scale, p.scale_t,
                  p.rows, p.cols, p.ld_x, p.ld_q, p.ld_scale, p.ld_qt, p.ld_scale_t,
                  (p.rows + 127) / 128, (p.cols + 127) / 128, e5m2 ? 57344.0f : 448.0f};
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(p.stream);
    return p.x_dtype == TR_DTYPE_F32 ? launch_in<float>(a, p.block_rows == 128, e5m2, stream)
                                     : launch_in<__nv_bfloat16>(a, p.block_rows == 128, e5m2, stream);
}

}  // namespace tr

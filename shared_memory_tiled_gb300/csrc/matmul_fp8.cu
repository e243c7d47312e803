// Matrix product of 8-bit operands with a scale for each block of 128 along
// the contraction.
//
// One operand, P, supplies the 128 rows of a tensor-core tile and the other,
// Q, its BN columns: P = a and Q = b, or, for a few rows of a, the other way
// round (TURN), so that they are the short side.  Per block of the contraction the tensor
// cores sum P Q^T in tensor memory; since the scales change with every block,
// four warps then take the sums out, multiply them by the block's scales and
// add them up in registers, while the next block's product runs into the other
// half of the tensor memory.
//
//   warp 0     TMA: keeps the ring of operand stages full
//   warp 1     matrix instructions, 4 per stage
//   warps 2-5  lane = row of P: sums += scale_p * scale_q * block sums
//
// Few tiles: the blocks of the contraction are split over a cluster of CTAs and
// their sums joined through distributed shared memory, in rank order.
//
// Measured on one GB300 (a bf16 library product reaches 1920 TFLOP/s there; 8-bit
// instructions run at twice its rate), ten calls in a row at 2070 MHz:
//   8192^3, 1x128 by 128x128 scales, bf16 out        427 us, 2.57 PFLOP/s
//     the same for a second on end (1930 MHz under the power cap)  458 us, 2.40 PFLOP/s
//   8192^3, 1x128 by 1x128                           600 us, 1.83 PFLOP/s
//   4096 x 2048 x 16384, 1x128 by 1x128, fp32 out    174 us, 1.58 PFLOP/s
//   2048^3                                          13.5 us, 1.27 PFLOP/s
//   777 x 2049 x 1111                               13.2 us
//   1, 16 and 64 x 8192 x 8192                14.1, 14.9, 19.0 us: 4.8, 4.5, 3.6 TB/s
//   with `accumulate`, 1x128 by 1x128, fp32: 8192^3 1471 us (618 without), 4096 x 2048 x
//     16384 293 us (174): the large tiles then read, add and write value by value
//
// What bounds the large ones is the exchange between the tensor cores and the warps
// that take the sums out, once for each block of 128: the instructions alone run at
// 250 us for 8192^3 from operands that are in place, at 322 us with the loads, but a
// warp's turn on a block takes 900 cycles in a row (its waits about 100 each, 400 for
// four reads of 32 columns with the additions between them, the rest for the scales,
// the hand back and the loop) and a buffer of sums, of which tensor memory holds
// two, goes through instructions and warps in turn.  With a scale to each column it is the
// multiplications and the reads of those scales as well: 0.67 us a block, 0.48 without.
#include <atomic>
#include <type_traits>

#include "bounds.cuh"
#include "launch.cuh"
#include "operand_ring.cuh"
#include "register_split.cuh"
#include "row_chunk.cuh"
#include "tcgen05.cuh"
#include "tensor_map.cuh"
#include "tr_internal.h"
#include "wait_selftest.cuh"

namespace tr {

// Set when a bounded in-kernel wait ran out; read and cleared by the host.
__device__ unsigned g_fault_flag_matmul = 0;

namespace {

constexpr int kThreads = 192;
constexpr int kBlockK = 128;             // bytes, values and the scales' block
constexpr int kTileP = 128;
constexpr int kBytesP = kTileP * kBlockK;

constexpr int kSumPitch = 132;           // words to a row of a tile's sums in shared memory

template <int BN>
struct Shape {
    static constexpr int kStageBytes = kBytesP + BN * kBlockK;
    // A tile of 16 columns is bound by P's bytes: four CTAs to an SM with 2 stages each
    // beat two with 5 (1 x 8192 x 8192: 14.5 against 16.1 us), since one's first
    // loads and last sums run beside the others' streams.
    static constexpr int kPerSm = BN == 16 ? 4 : 2;
    static constexpr int kStages = BN == 16 ? 2 : BN == 128 ? 3 : BN == 64 ? 4 : 5;
    static constexpr int kColumns = 2 * BN;  // two buffers of sums
    // Blocks whose scales are in shared memory or on their way.  Four to the small tile, whose
    // few blocks would wait for the first copies (1 x 4096 x 4096: 7.5 us, 7.7 with
    // eight); with four the larger ones wait for a block's copies (32 x 8192 x 8192:
    // 17.3 us, 16.4 with eight).
    static constexpr int kScaleSlots = BN == 16 ? 4 : 8;
    static constexpr size_t kSmem = 1024 + size_t(kStages) * kStageBytes;
};

struct Product {
    const float *scale_p, *scale_q;
    void *out;
    int64_t ld_p, ld_q, ld_out;          // pitches of the scales and of the output
    int64_t p, q;                        // rows of the two operands
    int64_t tiles_p, tiles_q;
    int32_t blocks;                      // blocks of the contraction
    int32_t split;                       // CTAs that share one tile's contraction
    int32_t p_block, q_block;            // rows to a scale: 1 or 128
    int32_t p_e5m2, q_e5m2;
    int32_t out_bf16, accumulate;
    // The least scale that the quantizer gives, which is that of a block of zeros: the sums
    // with it are zero, whatever the factor, or those of magnitudes up to 2^-100.
    float floor_p, floor_q;
};

// Rows of P and of Q at which a tile of bp x bq begins; `most` tiles of P go with
// each tile of Q before the next, so that the operands in use at one time stay
// in L2.  In 32 bits: there are fewer than 2^31 tiles, and a 64-bit division is a call, around
// which k_matmul_pair's warps with few registers would spill.
__device__ __forceinline__ void tile_at(const Product &g, int64_t tile, int bp, int bq, uint32_t most,
                                        int64_t *p0, int64_t *q0) {
    const uint32_t tiles_p = uint32_t(g.tiles_p), tiles_q = uint32_t(g.tiles_q);
    const uint32_t group = uint32_t(tile) / (most * tiles_q), at = uint32_t(tile) - group * most * tiles_q;
    const uint32_t left = tiles_p - group * most, tall = left < most ? left : most;
    *p0 = int64_t(group * most + at % tall) * bp;
    *q0 = int64_t(at / tall) * bq;
}

// out[i][j] = v, or += v; `s` is the output's logical extent.
__device__ __forceinline__ void put(const Product &g, int64_t i, int64_t j, float v,
                                    const dbg::Side &s) {
    if (g.out_bf16) {
        __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(g.out) + i * g.ld_out + j;
        if (!TR_STORE_OK(s, o, 2)) return;
        if (g.accumulate) v += __bfloat162float(*o);
        *o = __float2bfloat16_rn(v);
    } else {
        float *o = static_cast<float *>(g.out) + i * g.ld_out + j;
        if (!TR_STORE_OK(s, o, 4)) return;
        if (g.accumulate) v += *o;
        *o = v;
    }
}

// The same for four neighbouring values on a boundary of their size together.
__device__ __forceinline__ void put4(const Product &g, int64_t i, int64_t j, float (&v)[4], const dbg::Side &s) {
    if (g.out_bf16) {
        uint2 *o = reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(g.out) + i * g.ld_out + j);
        if (!TR_STORE_OK(s, o, 8)) return;
        if (g.accumulate) {
            const uint2 old = *o;
            v[0] += __uint_as_float(old.x << 16);
            v[1] += __uint_as_float(old.x & 0xffff0000u);
            v[2] += __uint_as_float(old.y << 16);
            v[3] += __uint_as_float(old.y & 0xffff0000u);
        }
        const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
        *o = make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
    } else {
        float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(g.out) + i * g.ld_out + j);
        if (!TR_STORE_OK(s, o, 16)) return;
        float4 old = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (g.accumulate) old = *o;
        *o = make_float4(v[0] + old.x, v[1] + old.y, v[2] + old.z, v[3] + old.w);
    }
}

// Least (zeros left out) and largest magnitude of some scales, as bits, which order alike
// (a NaN is the largest); `least` one lower, so that a zero is the largest number there.
struct ScaleRange {
    uint32_t below_least, most;
    __device__ __forceinline__ void add(float v) {
        const uint32_t m = __float_as_uint(v) & 0x7fffffffu;
        below_least = min(below_least, m - 1);
        most = max(most, m);
    }
    __device__ __forceinline__ void add_but(float floor, float v) {
        if (v != floor) add(v);
    }
    __device__ __forceinline__ void join_warp() {
        below_least = __reduce_min_sync(0xffffffffu, below_least);
        most = __reduce_max_sync(0xffffffffu, most);
    }
    __device__ __forceinline__ float least() const { return __uint_as_float(below_least + 1); }
    __device__ __forceinline__ float largest() const { return __uint_as_float(most); }
};
constexpr uint32_t kNoneYet = 0x7f7fffffu;  // below infinity: no factor is small with it

// Whether the product of two scales of these ranges may leave the normal numbers of 32 bits.
__device__ __forceinline__ bool out_of_range(const ScaleRange &a, const ScaleRange &b) {
    return a.largest() * b.largest() > 3.402823466e38f || a.least() * b.least() < 1.175494351e-38f;
}

// A row's scale where its product with the columns' scales leaves the normal numbers:
// block sums are below 2^39 and, if not zero, above 2^-33, so sums times two such scales
// may well be finite, and zero times both is zero.  A power of two then moves from the
// scale to `pre`, which multiplies the sums first; both steps are exact while a block's
// column scales are within 2^190 of one another.  Elsewhere `pre` is 1.  The bits are
// those of the plain factor wherever that is in range.
//
// Such blocks have a loop of their own, and what finds them stays out of the way of the
// warps that add: in the pair kernel the warps that copy the scales take a batch's range
// (and copy with few instructions, since a late batch stops everything), in the other
// each thread looks at its own two scales a block ahead.  A look at the block in hand,
// with both forms of the sum behind a branch, took 8192^3 from 433 to 477 us (1x128 by
// 1x128: 621 to 727); so it is 428 (600).  Blocks of zeros, as masked rows have, do not
// count: with them a tenth of the rows zero in e5m2 took 591 us, without 430.
struct RowScale {
    float f, pre;
};
__device__ __forceinline__ RowScale row_scale(float sp, float floor, const ScaleRange &q) {
    const float m = fabsf(sp);
    if (m * q.largest() > 3.402823466e38f) return RowScale{sp * 0x1p-60f, 0x1p60f};
    if (m != 0.0f && m != floor && m * q.least() < 1.175494351e-38f) return RowScale{sp * 0x1p60f, 0x1p-60f};
    return RowScale{sp, 1.0f};
}
// The range of N columns' scales (0: of the one that they share), for row_scale.
template <int N>
__device__ __forceinline__ ScaleRange column_range(const float *q, float floor, int lane) {
    ScaleRange r{kNoneYet, 0};
    if constexpr (N == 0) {
        r.add_but(floor, q[0]);
    } else {
#pragma unroll
        for (int c = lane; c < N; c += 32) r.add_but(floor, q[c]);
        r.join_warp();
    }
    return r;
}

// Adds up the sums of a tile that SPLIT CTAs left in shared memory, in rank order, and
// writes this CTA's share of the tile.  Eight loads go out before the first is
// used: one from another CTA takes some 450 cycles (one at a time they were
// three quarters of a 2048^3 product).
template <int BN, bool TURN, int SPLIT>
__device__ __forceinline__ void store_tile(const Product &g, const float *red, int64_t p0, int64_t q0, int rank,
                                           int th, const dbg::Side &s) {
    uint32_t base[SPLIT];
#pragma unroll
    for (int peer = 0; peer < SPLIT; ++peer) base[peer] = ptx::peer_addr(red, uint32_t(SPLIT == 1 ? rank : peer));
    if constexpr (TURN) {
        // Threads along the rows of P (neighbouring columns of the output), 8 / SPLIT
        // rows of the output at a time.
        constexpr int U = 8 / SPLIT;
        for (int c0 = rank; c0 < BN && q0 + c0 < g.q; c0 += SPLIT * U) {
            float v[U][SPLIT];
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int peer = 0; peer < SPLIT; ++peer)
                    v[u][peer] = ptx::load_cluster(base[peer] + 4 * ((c0 + u * SPLIT) % BN * 128 + th));
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int c = c0 + u * SPLIT;
#pragma unroll
                for (int peer = 1; peer < SPLIT; ++peer) v[u][0] += v[u][peer];
                if (c < BN && q0 + c < g.q && p0 + th < g.p) put(g, q0 + c, p0 + th, v[u][0], s);
            }
        }
    } else {
        // A warp takes rows of the tile: 4 neighbouring columns to a lane where they can
        // be stored at once, else every 32nd.
        constexpr int ROWS = 32 / SPLIT, U = ROWS < 8 ? ROWS : 8, PEERS = 8 / U;
        const int lane = th & 31, es = g.out_bf16 ? 2 : 4;
        const bool whole = q0 + BN <= g.q && g.ld_out % 4 == 0 && reinterpret_cast<uintptr_t>(g.out) % (4 * es) == 0;
#pragma unroll 1
        for (int i = 0; i < ROWS; i += U) {
            auto row = [&](int u) { return ((i + u) * SPLIT + rank) * 4 + (th >> 5); };
            float v[U][4] = {};
#pragma unroll
            for (int peer = 0; peer < SPLIT; peer += PEERS) {
                float4 t[PEERS][U];
#pragma unroll
                for (int k = 0; k < PEERS; ++k)
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        const uint32_t at = base[peer + k] + 4 * (row(u) * kSumPitch);
                        if (whole) {
                            t[k][u] = ptx::load_cluster4(at + 16 * lane);
                        } else {
                            t[k][u].x = ptx::load_cluster(at + 4 * lane);
                            t[k][u].y = ptx::load_cluster(at + 4 * lane + 128);
                            t[k][u].z = ptx::load_cluster(at + 4 * lane + 256);
                            t[k][u].w = ptx::load_cluster(at + 4 * lane + 384);
                        }
                    }
#pragma unroll
                for (int k = 0; k < PEERS; ++k)
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        v[u][0] += t[k][u].x;
                        v[u][1] += t[k][u].y;
                        v[u][2] += t[k][u].z;
                        v[u][3] += t[k][u].w;
                    }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t r = p0 + row(u);
                if (r >= g.p) continue;
                if (whole) {
                    put4(g, r, q0 + lane * 4, v[u], s);
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (q0 + lane + k * 32 < g.q) put(g, r, q0 + lane + k * 32, v[u][k], s);
                }
            }
        }
    }
}

template <int BN, bool TURN, bool QROW>
__global__ void __launch_bounds__(kThreads, Shape<BN>::kPerSm)
k_matmul_fp8(const __grid_constant__ CUtensorMap map_p, const __grid_constant__ CUtensorMap map_q,
             const __grid_constant__ Product g) {
    using S = Shape<BN>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t full[S::kStages], empty[S::kStages], sums_full[2], sums_empty[2], drained;
    __shared__ uint32_t tmem_base;
    // Scales, all slots but one ahead: each of the 128 threads copies its row's of P and one
    // of Q (QROW: a column's; else all the same one, each its own copy).
    __shared__ alignas(16) float scales_p[S::kScaleSlots][128], scales_q[S::kScaleSlots][128];
    uint8_t *stages = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;

    if (t == 0) {
        ptx::prefetch_tensormap(&map_p);
        ptx::prefetch_tensormap(&map_q);
        for (int i = 0; i < S::kStages; ++i) {
            ptx::mbar_init(full + i, 1);
            ptx::mbar_init(empty + i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(sums_full + i, 1);
            ptx::mbar_init(sums_empty + i, 4);
        }
        ptx::mbar_init(&drained, 1);
        ptx::fence_barrier_init();
    }
    if (warp == 1) ptx::tmem_alloc(&tmem_base, S::kColumns);
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = tmem_base;
    // The dependents may start once every block has its tensor memory: one that
    // waited for columns held by a dependent would wait for ever.
    pdl_prologue();

    const int64_t tile = blockIdx.x / unsigned(g.split);
    const int rank = int(blockIdx.x % unsigned(g.split));
    int64_t p0, q0;
    tile_at(g, tile, kTileP, BN, 16, &p0, &q0);
    const int first = int(int64_t(g.blocks) * rank / g.split);
    const int count = int(int64_t(g.blocks) * (rank + 1) / g.split) - first;
    bool ok = true;

    float2 acc[BN / 2];
#pragma unroll
    for (int c = 0; c < BN / 2; ++c) acc[c] = make_float2(0.0f, 0.0f);

    if (warp == 0) {
        if (lane == 0) {
            int i = 0;
            for (; i < count; ++i) {
                const int s = i % S::kStages;
                if (i >= S::kStages && !ptx::mbar_wait_bounded(empty + s, ((i / S::kStages) - 1) & 1)) {
                    ok = false;
                    break;
                }
                uint8_t *dst = stages + s * S::kStageBytes;
                ptx::mbar_arrive_expect_tx(full + s, S::kStageBytes);
                ptx::tma_load_2d(dst, &map_p, full + s, (first + i) * kBlockK, int32_t(p0));
                ptx::tma_load_2d(dst + kBytesP, &map_q, full + s, (first + i) * kBlockK, int32_t(q0));
            }
            // Nothing may arrive after the block has gone.
            if (!leave_ring<S::kStages>(
                    i, [&](int s, uint32_t parity) { return ptx::mbar_wait_bounded(empty + s, parity); },
                    [&](int s, uint32_t parity) { ptx::mbar_wait_bounded(full + s, parity); }))
                ok = false;
        }
    } else if (warp == 1) {
        // The whole warp goes through the loop and one elected lane issues, which leaves
        // the descriptors in uniform registers: see k_matmul_pair.
        const bool leader = ptx::elect_one();
        const uint32_t idesc = ptx::f8_idesc(g.p_e5m2, g.q_e5m2, 128, BN);
        for (int i = 0; i < count; ++i) {
            const int s = i % S::kStages, b = i & 1;
            ok = ptx::mbar_wait_bounded(full + s, (i / S::kStages) & 1) &&
                 (i < 2 || ptx::mbar_wait_bounded(sums_empty + b, ((i >> 1) - 1) & 1));
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            ptx::tc_fence_after();
            const uint32_t at = ptx::smem_addr(stages + s * S::kStageBytes);
            const uint64_t dp = ptx::operand_desc(at), dq = ptx::operand_desc(at + kBytesP);
            if (leader) {
#pragma unroll
                for (int k = 0; k < kBlockK / 32; ++k)
                    ptx::mma_f8(tmem + b * BN, dp + 2 * k, dq + 2 * k, idesc, k > 0);
                ptx::mma_commit(sums_full + b);
                ptx::mma_commit(empty + s);
            }
        }
        if (!ok) {
            if (leader) ptx::mma_commit(&drained);
            ptx::mbar_wait_bounded(&drained, 0);
        }
    } else {
        const int w = warp & 3;                       // the quarter of the lanes this warp may read
        const int row = w * 32 + lane, th = t - 64;   // row of P; index among the 128 threads
        const int64_t col = q0 + (QROW ? th : 0);     // whose scale this thread takes
        const bool has_p = p0 + row < g.p, has_q = (!QROW || th < BN) && col < g.q;
        const float *sp = g.scale_p + (g.p_block == 1 ? p0 + row : (p0 + row) >> 7);
        const float *sq = g.scale_q + (g.q_block == 1 ? col : col >> 7);
        [[maybe_unused]] const dbg::Side side_p = dbg::side(g.scale_p, 1, g.blocks, g.p_block == 1 ? g.p : (g.p + 127) / 128, g.ld_p, 0, 4);
        [[maybe_unused]] const dbg::Side side_q = dbg::side(g.scale_q, 1, g.blocks, g.q_block == 1 ? g.q : (g.q + 127) / 128, g.ld_q, 0, 4);
        auto copy_scales = [&](int i) {
            const float *p = sp + int64_t(first + i) * g.ld_p, *q = sq + int64_t(first + i) * g.ld_q;
            const bool now = i < count;
            ptx::cp_async_4_or_zero(&scales_p[i % S::kScaleSlots][th], now && has_p ? p : g.scale_p, now && has_p && TR_LOAD_OK(side_p, p, 4));
            ptx::cp_async_4_or_zero(&scales_q[i % S::kScaleSlots][th], now && has_q ? q : g.scale_q, now && has_q && TR_LOAD_OK(side_q, q, 4));
            ptx::cp_async_commit();
        };
        for (int i = 0; i < S::kScaleSlots - 1; ++i) copy_scales(i);
        // Whether block i's factors may leave the range, from this thread's own two scales:
        // by their product, or (QROW, where each meets the others') one by one.
        auto strays = [&](int i) {
            const float a = fabsf(scales_p[i % S::kScaleSlots][th]), b = fabsf(scales_q[i % S::kScaleSlots][th]);
            const bool some_a = a != 0.0f && a != g.floor_p, some_b = b != 0.0f && b != g.floor_q;
            if constexpr (QROW) return a > 0x1p63f || b > 0x1p63f || (a < 0x1p-63f && some_a) || (b < 0x1p-63f && some_b);
            return a * b > 3.402823466e38f || (a * b < 1.175494351e-38f && some_a && some_b);
        };
        ptx::cp_async_wait<S::kScaleSlots - 2>();
        bool apart = QROW ? ptx::named_any(1, 128, strays(0)) : __any_sync(0xffffffffu, strays(0));
        // Adds block i's sums; `first`: with factors that may leave the range.
        auto take = [&](int i, auto first) {
            const int b = i & 1, slot = i % S::kScaleSlots;
            ptx::cp_async_wait<S::kScaleSlots - 3>();  // this thread's copies for block i + 1 are here
            // Everybody's are, and block i - 1's are read.
            if constexpr (QROW) apart = ptx::named_any(1, 128, strays(i + 1));
            const float own_p = scales_p[slot][th], all_q = QROW ? 1.0f : scales_q[slot][th];
            float f = own_p * all_q;
            [[maybe_unused]] float pre = 1.0f;
            if constexpr (decltype(first)::value) {
                const RowScale own = row_scale(own_p, g.floor_p, column_range<QROW ? BN : 0>(&scales_q[slot][QROW ? 0 : th], g.floor_q, lane));
                f = own.f * all_q;
                pre = own.pre;
            }
            const float2 f2 = make_float2(f, f);
            copy_scales(i + S::kScaleSlots - 1);
            // A wait that ran out is not repeated, but the meetings go on.
            if (ok) ok = ptx::mbar_wait_bounded(sums_full + b, (i >> 1) & 1);
            __syncwarp();
            ptx::tc_fence_after();
            const uint32_t from = tmem + (uint32_t(w * 32) << 16) + b * BN;
            float v[2][16];
            ptx::tmem_load16(v[0], from);
#pragma unroll
            for (int c = 0; c < BN / 16; ++c) {
                ptx::tmem_wait_load16(v[c & 1]);
                if (c + 1 < BN / 16) {
                    ptx::tmem_load16(v[(c + 1) & 1], from + (c + 1) * 16);
                } else {  // every sum is in registers: the tensor cores may go on
                    ptx::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive_relaxed(sums_empty + b);
                }
                if constexpr (decltype(first)::value) {
#pragma unroll
                    for (int k = 0; k < 16; k += 2) {
                        const float2 two = __fmul2_rn(make_float2(v[c & 1][k], v[c & 1][k + 1]), make_float2(pre, pre));
                        v[c & 1][k] = two.x;
                        v[c & 1][k + 1] = two.y;
                    }
                }
#pragma unroll
                for (int k = 0; k < 16; k += 4) {
                    float2 f01 = f2, f23 = f2;
                    if constexpr (QROW) {
                        const float4 q = *reinterpret_cast<const float4 *>(&scales_q[slot][c * 16 + k]);
                        f01 = __fmul2_rn(f2, make_float2(q.x, q.y));
                        f23 = __fmul2_rn(f2, make_float2(q.z, q.w));
                    }
                    float2 &a0 = acc[c * 8 + k / 2], &a1 = acc[c * 8 + k / 2 + 1];
                    a0 = __ffma2_rn(make_float2(v[c & 1][k], v[c & 1][k + 1]), f01, a0);
                    a1 = __ffma2_rn(make_float2(v[c & 1][k + 2], v[c & 1][k + 3]), f23, a1);
                }
            }
            if constexpr (!QROW && !decltype(first)::value) apart = __any_sync(0xffffffffu, strays(i + 1));
        };
        int i = 0;
        for (; i < count && !apart; ++i) take(i, std::false_type());
        for (; i < count; ++i) take(i, std::true_type());  // the rest of the tile with it
        ptx::cp_async_wait_all();
        // The sums go through shared memory (the stages are free: every product is
        // complete) so that lanes write neighbouring words of the output.
        float *red = reinterpret_cast<float *>(stages);
        if constexpr (TURN) {
#pragma unroll
            for (int c = 0; c < BN / 2; ++c) {
                red[2 * c * 128 + row] = acc[c].x;
                red[(2 * c + 1) * 128 + row] = acc[c].y;
            }
        } else {
#pragma unroll
            for (int c = 0; c < BN / 4; ++c)
                *reinterpret_cast<float4 *>(red + row * kSumPitch + 4 * c) =
                    make_float4(acc[2 * c].x, acc[2 * c].y, acc[2 * c + 1].x, acc[2 * c + 1].y);
        }
    }
    if (!ok) atomicExch(&g_fault_flag_matmul, 1u);
    __syncwarp();
    ptx::tc_fence_before();
    __syncthreads();
    if (g.split > 1) ptx::cluster_sync();
    if (warp >= 2) {
        const int th = t - 64;
        [[maybe_unused]] const dbg::Side so = dbg::side(g.out, 1, TURN ? g.q : g.p, TURN ? g.p : g.q, g.ld_out, 0, g.out_bf16 ? 2 : 4);
        const float *red = reinterpret_cast<const float *>(stages);
        switch (g.split) {
            case 1: store_tile<BN, TURN, 1>(g, red, p0, q0, rank, th, so); break;
            case 2: store_tile<BN, TURN, 2>(g, red, p0, q0, rank, th, so); break;
            case 4: store_tile<BN, TURN, 4>(g, red, p0, q0, rank, th, so); break;
            default: store_tile<BN, TURN, 8>(g, red, p0, q0, rank, th, so); break;
        }
    }
    if (g.split > 1) ptx::cluster_sync();  // no block leaves while another reads its sums
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_free(tmem, S::kColumns);
    }
}

// --- large products: two CTAs to a 256 x 256 tile --------------------------------------
//
// A CTA pair loads 64 KB per block of the contraction for a 256 x 256 tile, 64 bytes
// a clock and SM at the tensor cores' full rate, half of what two 128 x 128 tiles
// would take from L2 and shared memory.  Resident pairs walk the tiles.  Per CTA:
//
//   warp 0     TMA of its 128 rows of P and of its half of Q
//   warp 1     (rank 0) matrix instructions of both CTAs, 4 per stage
//   warps 2, 3 scales of P and of Q, a batch of blocks ahead, and the batch's range
//   warps 4-11 two groups of 128 threads, 128 columns each: a thread takes its row's
//              block sums out of tensor memory, 32 columns at a time with the next
//              32 on the way, and adds them, scaled, to 128 sums in registers
//
// QROW: Q has a scale to each row (a column of the tile): its 128 scales go through
// shared memory; else one scale for the group's columns, and one multiplication
// fewer to each value.

constexpr int kPairTile = 256;
// Blocks whose scales come together, with one notice each way: 8192^3 takes 436 us with
// batches of 8, 470 with a notice each way for every block.
constexpr int kBatch = 8;
constexpr int kPairStages = 5;
constexpr int kPairStageBytes = 2 * kBytesP;       // 128 rows of P and 128 of Q
constexpr int kStagingBytes = 8 * 32 * 128;        // 32 rows of 128 bytes to each of 8 warps
constexpr size_t kPairSmem = 1024 + size_t(kPairStages) * kPairStageBytes + kStagingBytes;

// Writes 32 rows x 128 columns from registers: a thread holds a row's sums, lanes
// write 128-byte pieces of rows.  The staging tile's 16-byte chunks stand at chunk
// XOR row % 8, so that neither side shares a bank.
template <typename F>
__device__ __forceinline__ void store_rows(const Product &g, int64_t row0, int64_t col0, uint4 *staging,
                                           const F &value, const dbg::Side &s) {
    const int lane = threadIdx.x & 31;
    const int es = g.out_bf16 ? 2 : 4;
    const bool whole = !g.accumulate && col0 + 128 <= g.q && (g.ld_out * es) % 16 == 0 &&
                       (reinterpret_cast<uintptr_t>(g.out) & 15u) == 0;
    if (whole && g.out_bf16) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            __syncwarp();
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                uint32_t w[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int j = half * 64 + c * 8 + 2 * k;
                    const __nv_bfloat162 h = __floats2bfloat162_rn(value(j), value(j + 1));
                    w[k] = *reinterpret_cast<const uint32_t *>(&h);
                }
                staging[lane * 8 + (c ^ (lane & 7))] = make_uint4(w[0], w[1], w[2], w[3]);
            }
            __syncwarp();
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int r = k * 4 + (lane >> 3), c = lane & 7;
                __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(g.out) + (row0 + r) * g.ld_out + col0 + half * 64 + c * 8;
                if (row0 + r < g.p && TR_STORE_OK(s, o, 16))
                    *reinterpret_cast<uint4 *>(o) = staging[r * 8 + (c ^ (r & 7))];
            }
        }
        return;
    }
#pragma unroll
    for (int quarter = 0; quarter < 4; ++quarter) {
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const int j = quarter * 32 + c * 4;
            staging[lane * 8 + (c ^ (lane & 7))] =
                make_uint4(__float_as_uint(value(j)), __float_as_uint(value(j + 1)),
                           __float_as_uint(value(j + 2)), __float_as_uint(value(j + 3)));
        }
        __syncwarp();
        if (whole) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int r = k * 4 + (lane >> 3), c = lane & 7;
                float *o = static_cast<float *>(g.out) + (row0 + r) * g.ld_out + col0 + quarter * 32 + c * 4;
                if (row0 + r < g.p && TR_STORE_OK(s, o, 16))
                    *reinterpret_cast<uint4 *>(o) = staging[r * 8 + (c ^ (r & 7))];
            }
        } else {
            const float *f = reinterpret_cast<const float *>(staging);
            const int64_t col = col0 + quarter * 32 + lane;
            for (int r = 0; r < 32 && row0 + r < g.p; ++r)
                if (col < g.q) put(g, row0 + r, col, f[(r * 8 + ((lane >> 2) ^ (r & 7))) * 4 + (lane & 3)], s);
        }
    }
}

template <bool QROW>
__global__ void __launch_bounds__(kPairThreads, 1)
k_matmul_pair(const __grid_constant__ CUtensorMap map_p, const __grid_constant__ CUtensorMap map_q,
              const __grid_constant__ Product g) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t full[kPairStages], empty[kPairStages], sums_full[2], sums_empty[2];
    // Scales of two batches of blocks; one notice each way to a batch.
    __shared__ uint64_t scales_full[2], scales_empty[2];
    __shared__ uint32_t tmem_base;
    __shared__ alignas(16) float scales_p[2 * kBatch][128], scales_q[2 * kBatch][QROW ? 256 : 4];
    __shared__ ScaleRange ranges[2][2];  // of a batch's scales of P and of Q
    uint8_t *stages = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint4 *staging = reinterpret_cast<uint4 *>(stages + kPairStages * kPairStageBytes);
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const uint32_t rank = ptx::cluster_rank();

    if (t == 0) {
        ptx::prefetch_tensormap(&map_p);
        ptx::prefetch_tensormap(&map_q);
        for (int i = 0; i < kPairStages; ++i) {
            ptx::mbar_init(full + i, 1);
            ptx::mbar_init(empty + i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(sums_full + i, 1);
            ptx::mbar_init(sums_empty + i, 16);  // the warps of both CTAs
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(scales_full + i, 2);   // those of P and of Q
            ptx::mbar_init(scales_empty + i, 8);  // this CTA's warps
        }
        ptx::fence_barrier_init();
    }
    if (warp == 1) ptx::tmem_alloc_pair(&tmem_base, 512);
    ptx::tc_fence_before();
    __syncthreads();
    ptx::cluster_sync();  // the other CTA's barriers are ready
    ptx::tc_fence_after();
    const uint32_t tmem = tmem_base;
    pdl_prologue();  // after the tensor memory is taken, as above

    const int64_t tiles = g.tiles_p * g.tiles_q;
    const int64_t pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    bool ok = true;

    if (warp < 4) {
        ptx::registers_down<kFewRegisters>();
        if (warp == 0) {
            if (lane == 0) {
                int s = 0;
                int64_t filled = 0;
                uint32_t phase = 1;  // the first round finds every stage empty
                for (int64_t tile = pair; tile < tiles && ok; tile += pairs) {
                    int64_t p0, q0;
                    tile_at(g, tile, kPairTile, kPairTile, 8, &p0, &q0);
                    for (int i = 0; i < g.blocks; ++i) {
                        if (!ptx::mbar_wait_bounded(empty + s, phase)) {
                            ok = false;
                            break;
                        }
                        uint8_t *dst = stages + s * kPairStageBytes;
                        if (rank == 0) ptx::mbar_arrive_expect_tx(full + s, 2 * kPairStageBytes);
                        const uint32_t bar = ptx::peer_addr(full + s, 0);
                        ptx::tma_load_2d_pair(dst, &map_p, bar, i * kBlockK, int32_t(p0) + int32_t(rank) * 128);
                        ptx::tma_load_2d_pair(dst + kBytesP, &map_q, bar, i * kBlockK, int32_t(q0) + int32_t(rank) * 128);
                        ++filled;
                        if (++s == kPairStages) {
                            s = 0;
                            phase ^= 1;
                        }
                    }
                }
                // Nothing may arrive after the block has gone: the commits come to both CTAs,
                // each waits for its own.
                if (!leave_ring<kPairStages>(
                        filled, [&](int st, uint32_t parity) { return ptx::mbar_wait_bounded(empty + st, parity); },
                        [](int, uint32_t) {}))
                    ok = false;
                // Where one does not come there may be loads in flight, which complete on rank 0's
                // barriers: both CTAs give them many times the microseconds that they take.
                if (!ok) {
                    const uint64_t t0 = ptx::global_timer_ns();
                    for (uint32_t n = 0; n < 1u << 24 && ptx::global_timer_ns() - t0 < 2000000; ++n) {
                    }
                }
            }
        } else if (warp == 1) {
            if (rank == 0) {
                // The whole warp goes through the loop and one elected lane issues: the
                // compiler then keeps descriptors and addresses in uniform registers.
                // Inside `lane == 0` alone the four instructions of a block took 350
                // cycles to issue and the loop 1040, which bounded the kernel (8192^3:
                // 503 us against 470); now they take 120.
                const bool leader = ptx::elect_one();
                const uint32_t idesc = ptx::f8_idesc(g.p_e5m2, g.q_e5m2, 256, 256);
                int s = 0, b = 0;
                uint32_t phase = 0, sums_phase = 1;
                for (int64_t tile = pair; tile < tiles && ok; tile += pairs)
                    for (int i = 0; i < g.blocks; ++i) {
                        ok = ptx::mbar_wait_bounded(full + s, phase) && ptx::mbar_wait_bounded(sums_empty + b, sums_phase);
                        ok = __all_sync(0xffffffffu, ok);
                        if (!ok) break;
                        ptx::tc_fence_after();
                        const uint32_t at = ptx::smem_addr(stages + s * kPairStageBytes);
                        const uint64_t dp = ptx::operand_desc(at), dq = ptx::operand_desc(at + kBytesP);
                        const int used = s, into = b;
                        if (++s == kPairStages) {
                            s = 0;
                            phase ^= 1;
                        }
                        b ^= 1;
                        if (b == 0) sums_phase ^= 1;
                        if (leader) {
#pragma unroll
                            for (int k = 0; k < kBlockK / 32; ++k)
                                ptx::mma_f8_pair(tmem + into * 256, dp + 2 * k, dq + 2 * k, idesc, k > 0);
                            ptx::mma_commit_pair(sums_full + into);
                            ptx::mma_commit_pair(empty + used);
                        }
                    }
            }
        } else {
            // Scales, a batch of blocks ahead: warp 2 those of P, warp 3 those of Q.
            const bool of_p = warp == 2;
            const float *base = of_p ? g.scale_p : g.scale_q;
            const float floor = of_p ? g.floor_p : g.floor_q;
            const int64_t ld = of_p ? g.ld_p : g.ld_q, rows = of_p ? g.p : g.q;
            const int shift = (of_p ? g.p_block : g.q_block) == 1 ? 0 : 7;  // 2^shift rows to a scale
            // Scales to take, and the tile's rows from one to the next (block scales of P
            // are taken once for each row, those of Q once for each 128 columns).
            const int count = of_p ? 128 : QROW ? 256 : 2, apart = of_p || QROW ? 1 : 128;
            [[maybe_unused]] const dbg::Side side = dbg::side(base, 1, g.blocks, (rows + (1 << shift) - 1) >> shift, ld, 0, 4);
            float *ring = of_p ? &scales_p[0][0] : &scales_q[0][0];
            const int pitch = of_p ? 128 : QROW ? 256 : 4;
            // Blocks are counted through all tiles of this pair and copied by batches, one
            // batch ahead of the one in use.
            const uint32_t mine = pair < tiles ? uint32_t(tiles - 1 - pair) / uint32_t(pairs) + 1 : 0;
            const int64_t blocks = int64_t(mine) * g.blocks;
            int64_t tile = pair;
            int at = 0;         // the next block's place in its tile
            const float *row;   // the scale of its first row, and how many of `count` there are
            int have = 0;
            const int step = of_p && shift ? 0 : 1;  // from one scale to the next
            auto copy_batch = [&](int64_t first) {
                const int held = blocks - first < kBatch ? int(blocks - first) : kBatch;
                float *dst = ring + int(first % (2 * kBatch)) * pitch;
                for (int n = 0; n < held; ++n, dst += pitch) {
                    if (at == 0) {
                        int64_t p0, q0;
                        tile_at(g, tile, kPairTile, kPairTile, 8, &p0, &q0);
                        const int64_t r0 = of_p ? p0 + rank * 128 : q0, left = apart == 1 ? rows - r0 : (rows - r0 + 127) >> 7;
                        row = base + (r0 >> shift);
                        have = left < count ? int(left) : count;
                    }
                    for (int k = lane; k < count; k += 32) {
                        const float *p = row + k * step;
                        const bool in = k < have && TR_LOAD_OK(side, p, 4);
                        ptx::cp_async_4_or_zero(dst + k, in ? p : base, in);
                    }
                    row += ld;
                    if (++at == g.blocks) {
                        at = 0;
                        tile += pairs;
                    }
                }
            };
            copy_batch(0);
            int b = 0;           // of the batch in hand
            uint32_t phase = 1;  // of the other buffer's release, which the first batch finds free
            for (int64_t n = 0; n < blocks; n += kBatch) {
                ptx::cp_async_wait_all();
                __syncwarp();
                const int held = blocks - n < kBatch ? int(blocks - n) : kBatch;
                const float *batch = ring + b * kBatch * pitch;
                ScaleRange range{kNoneYet, 0};
                if (count == 2) {
                    if (lane < held) {
                        range.add(batch[lane * pitch]);
                        range.add(batch[lane * pitch + 1]);
                    }
                } else {
#pragma unroll 2
                    for (int k = lane * 4; k < held * count; k += 128) {  // count is the pitch
                        const float4 four = *reinterpret_cast<const float4 *>(batch + k);
                        range.add(four.x);
                        range.add(four.y);
                        range.add(four.z);
                        range.add(four.w);
                    }
                }
                range.join_warp();
                if (range.least() < 0x1p-90f) {  // blocks of zeros, most likely: again without them
                    range.below_least = kNoneYet;
#pragma unroll 1
                    for (int k = lane * 4; k < held * pitch; k += 128) {
                        const float4 four = *reinterpret_cast<const float4 *>(batch + k);
                        range.add_but(floor, four.x);
                        range.add_but(floor, four.y);
                        if (count == 2) continue;  // the other two words of that pitch hold nothing
                        range.add_but(floor, four.z);
                        range.add_but(floor, four.w);
                    }
                    range.join_warp();
                }
                if (lane == 0) ranges[b][of_p ? 0 : 1] = range;
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(scales_full + b);
                b ^= 1;
                if (n + kBatch < blocks) {
                    if (b == 0) phase ^= 1;
                    if (ok) ok = ptx::mbar_wait_bounded(scales_empty + b, phase);
                    copy_batch(n + kBatch);
                }
            }
        }
    } else {
        ptx::registers_up<kManyRegisters>();
        const int w = warp & 3, group = (warp - 4) >> 2, r = w * 32 + lane;
        const uint32_t tsum = tmem + (uint32_t(w * 32) << 16) + group * 128;
        const uint32_t release[2] = {ptx::peer_addr(sums_empty, 0), ptx::peer_addr(sums_empty + 1, 0)};
        [[maybe_unused]] const dbg::Side so = dbg::side(g.out, 1, g.p, g.q, g.ld_out, 0, g.out_bf16 ? 2 : 4);
        int b = 0, slot = 0;  // slot: of the block's scales
        uint32_t phase = 0, slot_phase = 0;
        bool apart = false;  // the batch has factors out of range
        for (int64_t tile = pair; tile < tiles; tile += pairs) {
            int64_t p0, q0;
            tile_at(g, tile, kPairTile, kPairTile, 8, &p0, &q0);
            p0 += rank * 128;
            q0 += group * 128;
            float2 acc[64];
#pragma unroll
            for (int c = 0; c < 64; ++c) acc[c] = make_float2(0.0f, 0.0f);
            float v[2][32];
            // Adds a block's sums; `first`: with factors that may leave the range of 32 bits.
            auto take = [&](auto first) {
                const float own_p = scales_p[slot][r], all_q = QROW ? 1.0f : scales_q[slot][group];
                float f = own_p * all_q;
                [[maybe_unused]] float pre = 1.0f;
                if constexpr (decltype(first)::value) {
                    ScaleRange cols{kNoneYet, 0};
                    if constexpr (QROW) {
#pragma unroll
                        for (int c = lane; c < 128; c += 32) cols.add(scales_q[slot][group * 128 + c]);
                        cols.join_warp();
                    } else {
                        cols.add(all_q);
                    }
                    const RowScale own = row_scale(own_p, 0.0f, cols);
                    f = own.f * all_q;
                    pre = own.pre;
                }
                const float2 f2 = make_float2(f, f);
                // Scales of the next 8 columns, read in this order: left to itself the
                // compiler reads each where it is used (8192^3: 640 us against 620; 16
                // columns ahead 637).
                [[maybe_unused]] float4 q_next[2];
                if constexpr (QROW) {
                    q_next[0] = ptx::load_shared_4(&scales_q[slot][group * 128]);
                    q_next[1] = ptx::load_shared_4(&scales_q[slot][group * 128 + 4]);
                }
                if (ok) ok = ptx::mbar_wait_bounded(sums_full + b, phase);
                __syncwarp();
                ptx::tc_fence_after();
                ptx::tmem_load32(v[0], tsum + b * 256);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    ptx::tmem_wait_load32(v[c & 1]);
                    if (c < 3) {
                        ptx::tmem_load32(v[(c + 1) & 1], tsum + b * 256 + (c + 1) * 32);
                    } else {  // every sum is in registers: the tensor cores may go on
                        ptx::tc_fence_before();
                        __syncwarp();
                        if (lane == 0) ptx::mbar_arrive_at(release[b]);
                    }
                    if constexpr (decltype(first)::value) {
#pragma unroll
                        for (int k = 0; k < 32; k += 2) {
                            const float2 two = __fmul2_rn(make_float2(v[c & 1][k], v[c & 1][k + 1]), make_float2(pre, pre));
                            v[c & 1][k] = two.x;
                            v[c & 1][k + 1] = two.y;
                        }
                    }
#pragma unroll
                    for (int k = 0; k < 32; k += 4) {
                        float2 f01 = f2, f23 = f2;
                        if constexpr (QROW) {
                            const int at = c * 32 + k;
                            const float4 q = q_next[k >> 2 & 1];
                            if (at + 8 < 128) q_next[k >> 2 & 1] = ptx::load_shared_4(&scales_q[slot][group * 128 + at + 8]);
                            f01 = __fmul2_rn(f2, make_float2(q.x, q.y));
                            f23 = __fmul2_rn(f2, make_float2(q.z, q.w));
                        }
                        float2 &a0 = acc[c * 16 + k / 2], &a1 = acc[c * 16 + k / 2 + 1];
                        a0 = __ffma2_rn(make_float2(v[c & 1][k], v[c & 1][k + 1]), f01, a0);
                        a1 = __ffma2_rn(make_float2(v[c & 1][k + 2], v[c & 1][k + 3]), f23, a1);
                    }
                }
                ++slot;
                b ^= 1;
                if (b == 0) phase ^= 1;
            };
            for (int i = 0; i < g.blocks;) {
                // The blocks of this tile that the batch in hand still holds.
                const int left = kBatch - slot % kBatch, end = i + left < g.blocks ? i + left : g.blocks;
                if (left == kBatch) {
                    // A wait that ran out is not repeated, but the arrivals go on.
                    if (ok) ok = ptx::mbar_wait_bounded(scales_full + slot / kBatch, slot_phase);
                    apart = out_of_range(ranges[slot / kBatch][0], ranges[slot / kBatch][1]);
                }
                if (apart) {
                    for (; i < end; ++i) take(std::true_type());
                } else {
                    for (; i < end; ++i) take(std::false_type());
                }
                if (slot % kBatch == 0) {
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(scales_empty + slot / kBatch - 1);  // its reads are done
                    if (slot == 2 * kBatch) {
                        slot = 0;
                        slot_phase ^= 1;
                    }
                }
            }
            store_rows(g, p0 + w * 32, q0, staging + (warp - 4) * 256,
                       [&](int j) { return j & 1 ? acc[j >> 1].y : acc[j >> 1].x; }, so);
        }
    }
    if (!ok) atomicExch(&g_fault_flag_matmul, 1u);
    __syncwarp();
    ptx::tc_fence_before();
    __syncthreads();
    ptx::cluster_sync();  // neither CTA leaves while the other's instructions read its operands
    ptx::tc_fence_after();
    if (warp == 1) ptx::tmem_free_pair(tmem, 512);
}

bool encode_operand(CUtensorMap *map, const void *base, int64_t k, int64_t rows, int64_t ld,
                    int box_rows) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {cuuint64_t(k), cuuint64_t(rows)};
    const cuuint64_t strides[1] = {cuuint64_t(ld)};
    const cuuint32_t box[2] = {kBlockK, cuuint32_t(box_rows)};
    const cuuint32_t estr[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box,
              estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Launches a kernel of this unit in clusters of `cluster` blocks, with its shared
// memory allowed once per device.
template <typename K>
cudaError_t launch_kernel(K kern, std::atomic<bool> *opted, int64_t grid, int threads, size_t smem, int cluster,
                          const CUtensorMap &map_p, const CUtensorMap &map_q, const Product &g,
                          cudaStream_t stream) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!opted[dev].load(std::memory_order_acquire)) {  // setting it twice is harmless
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
        if (e != cudaSuccess) return e;
        opted[dev].store(true, std::memory_order_release);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(grid));
    cfg.blockDim = dim3(unsigned(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = unsigned(cluster);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, kern, map_p, map_q, g);
    if (e != cudaSuccess) (void)cudaGetLastError();
    return e;
}

template <int BN, bool TURN, bool QROW>
cudaError_t launch_shape(const CUtensorMap &map_p, const CUtensorMap &map_q, const Product &g,
                         cudaStream_t stream) {
    static std::atomic<bool> opted[64];  // per device, zero-initialised (static)
    return launch_kernel(k_matmul_fp8<BN, TURN, QROW>, opted, g.tiles_p * g.tiles_q * g.split, kThreads,
                         Shape<BN>::kSmem, g.split, map_p, map_q, g, stream);
}

template <bool QROW>
cudaError_t launch_pair(const CUtensorMap &map_p, const CUtensorMap &map_q, const Product &g,
                        cudaStream_t stream) {
    static std::atomic<bool> opted[64], checked[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!checked[dev].load(std::memory_order_acquire)) {
        cudaFuncAttributes attr;
        e = cudaFuncGetAttributes(&attr, k_matmul_pair<QROW>);
        if (e != cudaSuccess) return e;
        if (!registers_suffice(attr.numRegs)) return cudaErrorLaunchOutOfResources;
        checked[dev].store(true, std::memory_order_release);
    }
    const int64_t pairs = sm_count() / 2, tiles = g.tiles_p * g.tiles_q;
    return launch_kernel(k_matmul_pair<QROW>, opted, 2 * (tiles < pairs ? tiles : pairs), kPairThreads, kPairSmem, 2,
                         map_p, map_q, g, stream);
}

__global__ void k_wait_selftest_matmul(int arrive, uint64_t limit_ns) {
    wait_selftest(&g_fault_flag_matmul, arrive, limit_ns);
}

}  // namespace

// Debug builds: this unit's record of refused accesses.
TR_BOUNDS_READER(read_bounds_matmul_fp8)

cudaError_t launch_wait_selftest_matmul(bool arrive, int64_t limit_ns, cudaStream_t stream) {
    k_wait_selftest_matmul<<<1, 32, 0, stream>>>(arrive ? 1 : 0, uint64_t(limit_ns));
    return cudaGetLastError();
}

cudaError_t read_and_clear_fault_matmul(unsigned *value) {
    cudaError_t e = cudaMemcpyFromSymbol(value, g_fault_flag_matmul, sizeof(unsigned));
    if (e != cudaSuccess) return e;
    const unsigned zero = 0;
    return cudaMemcpyToSymbol(g_fault_flag_matmul, &zero, sizeof(unsigned));
}

cudaError_t launch_matmul_fp8(const tr_matmul_fp8_args &a, const char **why) {
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(a.stream);
    const bool out_bf16 = a.out_dtype == TR_DTYPE_BF16;
    if (a.k == 0) {
        if (a.accumulate) return cudaSuccess;
        const size_t es = out_bf16 ? 2 : 4;
        return cudaMemset2DAsync(a.out, size_t(a.ld_out) * es, 0, size_t(a.n) * es, size_t(a.m), stream);
    }
    // Up to 64 rows of a: they are the columns of the tile, and b its 128 rows.
    const bool turn = a.m <= 64;
    // 256 x 256 tiles where 128 x 128 ones leave no room to split the contraction and no
    // side is inside one of them: 1280 x 2048 x 4096 (160 small tiles) takes 20.5 us on
    // the large and 26.4 on the small ones, 1280 x 1920 x 4096 (150) 24.7 and 18.6,
    // 192 x 65536 x 4096 72.6 and 95.9, 128 x 65536 x 4096 72.2 and 57.9.
    const bool pair = !turn && a.m > 128 && a.n > 128 &&
                      ((a.m + 127) / 128) * ((a.n + 127) / 128) > int64_t(sm_count());
    const int bn = pair ? 256 : !turn ? 128 : a.m <= 16 ? 16 : a.m <= 32 ? 32 : 64;
    Product g{};
    g.scale_p = turn ? a.scale_b : a.scale_a;
    g.scale_q = turn ? a.scale_a : a.scale_b;
    g.out = a.out;
    g.ld_p = turn ? a.ld_scale_b : a.ld_scale_a;
    g.ld_q = turn ? a.ld_scale_a : a.ld_scale_b;
    g.ld_out = a.ld_out;
    g.p = turn ? a.n : a.m;
    g.q = turn ? a.m : a.n;
    g.tiles_p = pair ? (g.p + 255) / 256 : (g.p + kTileP - 1) / kTileP;
    g.tiles_q = (g.q + bn - 1) / bn;
    g.blocks = int32_t((a.k + kBlockK - 1) / kBlockK);
    g.p_block = turn ? a.b_block_rows : a.a_block_rows;
    g.q_block = turn ? a.a_block_rows : a.b_block_rows;
    g.p_e5m2 = (turn ? a.b_dtype : a.a_dtype) == TR_DTYPE_E5M2;
    g.q_e5m2 = (turn ? a.a_dtype : a.b_dtype) == TR_DTYPE_E5M2;
    g.floor_p = g.p_e5m2 ? 0x1p-100f / 57344.0f : 0x1p-100f / 448.0f;
    g.floor_q = g.q_e5m2 ? 0x1p-100f / 57344.0f : 0x1p-100f / 448.0f;
    g.out_bf16 = out_bf16;
    g.accumulate = a.accumulate;
    // Split the contraction until the tiles fill what is resident at one time, each
    // CTA keeping four blocks or more.
    const int64_t tiles = g.tiles_p * g.tiles_q, resident = int64_t(sm_count()) * (bn == 16 ? Shape<16>::kPerSm : 2);
    g.split = 1;
    while (!pair && g.split < 8 && tiles * g.split * 2 <= resident && g.blocks >= g.split * 8)
        g.split *= 2;
    if (tiles * g.split > 0x7fffffffll) {
        *why = "matmul: too many tiles for one launch";
        return cudaErrorInvalidValue;
    }
    CUtensorMap map_a, map_b;
    if (!encode_operand(&map_a, a.a, a.k, a.m, a.lda, turn ? bn : kTileP) ||
        !encode_operand(&map_b, a.b, a.k, a.n, a.ldb, turn || pair ? kTileP : bn)) {
        *why = "matmul: cuTensorMapEncodeTiled rejected the operands (a pitch of 2^40 bytes or more)";
        return cudaErrorInvalidValue;
    }
    if (pair)
        return g.q_block == 1 ? launch_pair<true>(map_a, map_b, g, stream) : launch_pair<false>(map_a, map_b, g, stream);
#define TR_SHAPE(BN, TURN, P, Q)                                                   \
    return g.q_block == 1 ? launch_shape<BN, TURN, true>(P, Q, g, stream)          \
                          : launch_shape<BN, TURN, false>(P, Q, g, stream)
    if (!turn) TR_SHAPE(128, false, map_a, map_b);
    if (bn == 16) TR_SHAPE(16, true, map_b, map_a);
    if (bn == 32) TR_SHAPE(32, true, map_b, map_a);
    TR_SHAPE(64, true, map_b, map_a);
#undef TR_SHAPE
}

}  // namespace tr

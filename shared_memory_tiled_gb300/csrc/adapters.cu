// Low-rank adapters of many requests at once: out[i] = base[i] + B_g (scale_g A_g x_i) for
// each token i with its own adapter g.
//
// Bound by memory, 2 R (k + n) operations to 2 k + 4 n bytes of a token: x, base and out once, each adapter in use once.
// A plan, made once for a batch, puts the tokens in the order of their adapters and cuts them into tiles of up to 128; a
// cluster of CTAs works on a tile, contracts a part of k and makes a part of the columns each, and the inner values, which
// all of them need, go through distributed shared memory, never through memory.  They are summed in 32 bits and go into the
// second product as two bf16 terms, 16 significant bits against the output's 8 (three terms for fp32 outputs, 24 bits).
//   many tokens   k_adapters, tensor cores fed by TMA: 8192 tokens of 8 adapters, 8192 x 8192 rank 16, 64 and 128 70, 76
//                 and 85 us, 5.8, 5.5 and 5.1 TB/s (60, 62 and 64 at the copy rate); fp32 outputs, rank 64, 145 (102)
//   few tokens    k_adapters_few, matrix instructions of a warp straight from memory: bound by latency, three reads that
//                 wait for one another (plan, x and a, b); one token rank 16 and 64 7.2 and 13.0 us, 64 of 48 adapters
//                 15.5 and 36.3 (4.2 and 15.3 at the copy rate)
// How wide the launches are goes by the adapters that are registered, which the host knows, not by those in use: 8192
// tokens of 8 prompts, rank 16, take 73 us with 8 adapters registered, 101 with 64 and 100 with 2000.
// Two launches a call at the most; nothing depends on the order in which blocks run.
#include <type_traits>

#include "adapter_plan.cuh"
#include "launch.cuh"
#include "operand_ring.cuh"
#include "row_chunk.cuh"
#include "tcgen05.cuh"
#include "tensor_map.cuh"
#include "tr_internal.h"
#include "wait_selftest.cuh"

namespace tr {

// What went wrong (kFaultWait, kFaultPlan); read and cleared by the host.
__device__ unsigned g_fault_flag_adapters = 0;

namespace {

// --- the plan: tokens in the order of their adapters, cut into tiles -----------------------

constexpr int kPlanThreads = 1024;

// Counts, places and tiles in one block.  Each warp takes a run of neighbouring tokens and
// has counts of its own, so that the order is stable and nothing depends on timing:
//   1  a warp counts its tokens of each adapter (lanes with the same one are found together);
//   2  the counts become places: over the warps for each adapter, then over the adapters;
//   3  a warp walks its tokens again and puts them there.
__global__ void __launch_bounds__(kPlanThreads) k_adapter_plan(const int32_t *index, int32_t *plan, int tokens,
                                                               int adapters, int warps) {
    pdl_prologue();
    extern __shared__ int32_t counts[];  // [warps][adapters + 1]
    __shared__ int3 joined[32], carry;  // tokens, large tiles, small tiles
    const int groups = adapters + 1, t = threadIdx.x, lane = t & 31, warp = t >> 5;
    [[maybe_unused]] const dbg::Side si = dbg::side(index, 1, 1, tokens, tokens, 0, 4);
    [[maybe_unused]] const dbg::Side sp = dbg::side(plan, 1, 1, plan_bytes(tokens, adapters) / 4, plan_bytes(tokens, adapters) / 4, 0, 4);
    for (int i = t; i < warps * groups; i += kPlanThreads) counts[i] = 0;
    if (t == 0) carry = make_int3(0, 0, 0);
    __syncthreads();
    const int64_t run = ((int64_t(tokens) + warps - 1) / warps + 31) / 32 * 32;
    const int64_t first = warp * run, last = first + run < tokens ? first + run : tokens;
    auto group_of = [&](int64_t i) {
        const int32_t g = TR_LOAD_OK(si, index + i, 4) ? index[i] : -1;
        return g >= 0 && g < adapters ? g : adapters;
    };
    int32_t *mine = counts + warp * groups;
    auto walk = [&](auto put) {
        if (warp >= warps) return;
        constexpr int U = 8;  // loads on their way
        for (int64_t i0 = first; i0 < last; i0 += 32 * U) {
            int g[U];
#pragma unroll
            for (int u = 0; u < U; ++u) g[u] = i0 + u * 32 + lane < last ? group_of(i0 + u * 32 + lane) : 0;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (i0 + u * 32 >= last) break;
                const int64_t i = i0 + u * 32 + lane;
                const unsigned here = __ballot_sync(0xffffffffu, i < last);
                if (i < last) {
                    const unsigned same = __match_any_sync(here, g[u]);
                    put(i, g[u], __popc(same & ((1u << lane) - 1)));
                    __syncwarp(here);
                    if (lane == 31 - __clz(same)) mine[g[u]] += __popc(same);
                }
                __syncwarp();
            }
        }
    };
    walk([](int64_t, int, int) {});
    __syncthreads();
    // Tokens before each adapter, large tiles before it and small ones, 1024 adapters at a time.
    auto up = [&](int3 v) {  // sums over the lanes up to this one
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, v.x, o), y = __shfl_up_sync(0xffffffffu, v.y, o), z = __shfl_up_sync(0xffffffffu, v.z, o);
            if (lane >= o) v = make_int3(v.x + x, v.y + y, v.z + z);
        }
        return v;
    };
    const int64_t most = plan_tiles(tokens, adapters);
    for (int g0 = 0; g0 < groups; g0 += kPlanThreads) {
        const int g = g0 + t;
        int n = 0;
        if (g < groups)
            for (int w = 0; w < warps; ++w) n += counts[w * groups + g];
        const int rest = n % kPlanTile;
        const int3 own = make_int3(n, n / kPlanTile + (rest > kPlanFew), rest > 0 && rest <= kPlanFew);
        const int3 s = up(own);
        if (lane == 31) joined[warp] = s;
        __syncthreads();
        if (warp == 0) {
            const int3 was = joined[lane], j = up(was);
            joined[lane] = make_int3(carry.x + j.x - was.x, carry.y + j.y - was.y, carry.z + j.z - was.z);
            __syncwarp();
            if (lane == 31) carry = make_int3(carry.x + j.x, carry.y + j.y, carry.z + j.z);
        }
        __syncthreads();
        if (g < groups) {
            int at = joined[warp].x + s.x - own.x;
            const int64_t large = joined[warp].y + s.y - own.y, small = joined[warp].z + s.z - own.z;
            auto tile = [&](int64_t place, int from, int count) {
                int32_t *p = plan + plan_tiles_at() + 4 * place;
                if (TR_STORE_OK(sp, p, 16)) *reinterpret_cast<int4 *>(p) = make_int4(g, from, count, 0);
            };
            for (int k = 0; k < own.y; ++k) tile(large + k, at + k * kPlanTile, n - k * kPlanTile < kPlanTile ? n - k * kPlanTile : kPlanTile);
            if (own.z) tile(most - 1 - small, at + n - rest, rest);
            for (int w = 0; w < warps; ++w) {
                const int c = counts[w * groups + g];
                counts[w * groups + g] = at;
                at += c;
            }
        }
        __syncthreads();
    }
    int32_t *order = plan + plan_order_at(tokens, adapters);
    walk([&](int64_t i, int g, int before) {
        int32_t *p = order + mine[g] + before;
        if (TR_STORE_OK(sp, p, 4)) *p = int32_t(i);
    });
    if (t == 0 && TR_STORE_OK(sp, plan, 16)) *reinterpret_cast<int4 *>(plan) = make_int4(carry.y, tokens, adapters, carry.z);
}

// --- the adapters ---------------------------------------------------------------------------

// Plan, scale and base are read past L1 (__ldcg): k_adapters beside k_adapters_few reads them without a wait of its own.

// Tile k of a plan, of the large ones, the small ones or all; false where there is none.  A plan of other sizes has none,
// and is reported: its entries could be anything.
enum Which { kAll, kLarge, kSmall };
__device__ __forceinline__ bool plan_tile(const int32_t *plan, int64_t tokens, int64_t adapters, int which, int64_t k, int4 *tile) {
    const int4 head = __ldcg(reinterpret_cast<const int4 *>(plan));
    if (head.y != tokens || head.z != adapters) {
        if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(&g_fault_flag_adapters, kFaultPlan);
        return false;
    }
    const int64_t large = which == kSmall ? 0 : head.x, small = which == kLarge ? 0 : head.w;
    if (k >= large + small) return false;
    const int64_t place = k < large ? k : plan_tiles(tokens, adapters) - 1 - (k - large);
    *tile = __ldcg(reinterpret_cast<const int4 *>(plan + plan_tiles_at() + 4 * place));
    return true;
}

struct Adapt {
    const float *scale;
    const int32_t *plan;
    const void *base;
    void *out;
    int64_t tokens, adapters, n;
    int64_t ld_base, ld_out;
    int32_t rank, chunks;  // chunks of 64 of the contraction over k
    int32_t split;         // CTAs that share a tile
    int32_t which;         // tiles (Which)
    int32_t beside;        // the small ones are another kernel's, just before this one
};

// The bf16 terms that inner values go into the second product as, two values' in a word each: the leading 8 significant
// bits, cut off and not rounded, the next 8 (with three terms), and the rest rounded.  Two terms stand for 16 bits and three
// for all 24, in products with b that are exact in 32 bits.  Cut off, because the terms then have the value's sign and none
// is larger: with an infinite b each gives the infinity that the value gives (rounded, every second value is followed by a
// term of the other sign, and the sum is NaN), and a value above bf16's largest does not become infinite.  For the same
// reason no term of a value is zero: where nothing would be left for the next, it gets half (exact while that is not
// subnormal).  An infinity or NaN is every one of its terms.  The smallest comes first, as they are added: halves of a last bit
// make that bit before they meet the rest.
// Rounded terms take as long (8192 tokens, rank 64, 76.1 us, these 76.3; 64 tokens of 48 adapters 15.3 either way); three
// for bf16 outputs, 24 bits where 8 are kept, would cost one token rank 16 7.0 -> 7.8 us and 8192 rank 128 85 -> 118.
template <int TERMS>
__device__ __forceinline__ void terms_of(float a, float b, uint32_t (&word)[TERMS]) {
    float left[2] = {a, b};
#pragma unroll
    for (int term = 0; term + 1 < TERMS; ++term) {
        float cut[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            cut[i] = __uint_as_float(__float_as_uint(left[i]) & 0xffff0000u);
            if (cut[i] == left[i]) cut[i] = left[i] = 0.5f * left[i];
            else left[i] -= cut[i];
        }
        word[TERMS - 1 - term] = __byte_perm(__float_as_uint(cut[0]), __float_as_uint(cut[1]), 0x7632);
    }
    const __nv_bfloat162 two = __floats2bfloat162_rn(left[0], left[1]);
    word[0] = *reinterpret_cast<const uint32_t *>(&two);
}

constexpr int kGroups = 3;              // of four warps that take sums out of tensor memory, each with its own
constexpr int kThreads = 128 + 128 * kGroups;
constexpr int kTileX = 128 * 128;       // bytes of 128 rows x 64 values
constexpr int kColumns = 128;           // of the output, worked on together
constexpr int kBox = 32;                // neighbouring tokens' rows to a load
// Word c (a multiple of 4) of a row of inner values in shared memory: chunks of 16 bytes in an order that 8
// rows' accesses to the same chunk do not share a bank.
template <int RP>
__device__ __forceinline__ int inner_at(int row, int c) {
    return row * RP + ((c >> 2) ^ (RP == 16 ? row >> 1 & 3 : row & 7)) * 4;
}

// RP: the rank, filled up with zeros; TERMS: bf16 values to an inner value.
template <int RP, int TERMS>
struct Shape {
    static constexpr int kStageBytes = kTileX + RP * 128;            // of x and a, or a tile of b
    static constexpr int kHalves = RP > 32 ? 2 : 1;                  // groups of warps that share the inner values
    static constexpr int kInner = 128 * RP * 4, kTerms = (RP * TERMS + 63) / 64 * kTileX;
    // The terms have a place of their own where that costs few stages: the cluster need not meet again before they are
    // written.
    static constexpr bool kApart = RP <= 32;
    static constexpr int kRegion = kApart ? kInner + kTerms : kInner > kTerms ? kInner : kTerms, kTermsAt = kApart ? kInner : 0;
    // Of 224 KB: two slots of 16 KB for base to each group (they also hold what a warp exchanges where base does not
    // come through them), or one, and the rest for stages.  Before the inner values are there the slots are stages too.
    static constexpr int kRoom = 224 * 1024 - kRegion;
    static constexpr int kPer = kRoom - 2 * kGroups * kTileX >= 2 * kStageBytes ? 2 : 1;
    static constexpr int kSlots = kGroups * kPer;
    static constexpr int kStages = (kRoom - kSlots * kTileX) / kStageBytes < 6 ? (kRoom - kSlots * kTileX) / kStageBytes : 6;
    static constexpr int kStagesX = kRoom / kStageBytes < 12 ? kRoom / kStageBytes : 12;
    static constexpr size_t kSmem = 1024 + kRegion + size_t(kRoom);
    // One CTA to an SM: a second would wait for tensor memory that the first's cluster may need to go on.
    static_assert(kStages >= 2 && 2 * kSmem > 228 * 1024, "one CTA to an SM");
};

// Copies `count` rows of columns [j0, j1) from base to out, or zeros.
template <typename T>
__device__ __forceinline__ void copy_rows(const Adapt &g, const int32_t *rows, int count, int64_t j0, int64_t j1, bool whole,
                                          const dbg::Side &sb, const dbg::Side &so) {
    constexpr int V = 16 / int(sizeof(T));
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int r = warp; r < count; r += kThreads / 32) {
        const T *p = static_cast<const T *>(g.base) + rows[r] * g.ld_base;
        T *o = static_cast<T *>(g.out) + rows[r] * g.ld_out;
        constexpr int U = 8;  // loads on their way
        if (whole) {
            for (int64_t j = j0 + lane * V; j < j1; j += U * 32 * V) {
                uint4 v[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int64_t c = j + u * 32 * V;
                    v[u] = make_uint4(0u, 0u, 0u, 0u);
                    if (g.base && c < j1 && TR_LOAD_OK(sb, p + c, 16)) v[u] = __ldcg(reinterpret_cast<const uint4 *>(p + c));
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int64_t c = j + u * 32 * V;
                    if (c < j1 && TR_STORE_OK(so, o + c, 16)) *reinterpret_cast<uint4 *>(o + c) = v[u];
                }
            }
        } else {
            for (int64_t j = j0 + lane; j < j1; j += U * 32) {
                T v[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int64_t c = j + u * 32;
                    v[u] = g.base && c < j1 && TR_LOAD_OK(sb, p + c, int(sizeof(T))) ? __ldcg(p + c) : T(0.0f);
                }
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (j + u * 32 < j1 && TR_STORE_OK(so, o + j + u * 32, int(sizeof(T)))) o[j + u * 32] = v[u];
            }
        }
    }
}

// One tile of up to 128 tokens of one adapter to a cluster.  Each CTA contracts its part of k on the tensor
// cores, D[token][r] = X A^T; the parts are joined through distributed shared memory, in rank order, each CTA
// joining some of the tokens and fetching the others; then each CTA makes its part of the output's columns,
// D[token][column] = V B^T, 128 at a time, with the inner values V in TERMS bf16 terms.
//
//   warp 0     TMA: keeps the ring full, first with x and a, then with b
//   warp 1     matrix instructions
//   warp 2     TMA: keeps the slots full with pieces of base, 128 rows x 128 bytes in the 128-byte swizzle
//   warps 4-   groups of four that take the tiles of columns in turn, lane = token: inner values (the first groups),
//              then base + sums in a piece's place, and from there rows of 128 bytes to out
//
// EDGE: rows of base and out that are off 16-byte boundaries or end off them.
template <int RP, typename T, bool EDGE>
__global__ void __launch_bounds__(kThreads, 1)
k_adapters(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_x32, const __grid_constant__ CUtensorMap map_rows,
           const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
           const __grid_constant__ CUtensorMap map_base, const __grid_constant__ CUtensorMap map_base32, const __grid_constant__ CUtensorMap map_base_rows,
           const __grid_constant__ Adapt g) {
    constexpr int TERMS = sizeof(T) == 2 ? 2 : 3;
    using S = Shape<RP, TERMS>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t full_x[S::kStagesX], empty_x[S::kStagesX], full[S::kStages], empty[S::kStages];
    __shared__ uint64_t joined[3], inner_full, inner_ready, sums_full[kGroups], sums_empty[kGroups], drained;
    __shared__ uint64_t base_full[S::kSlots], base_empty[S::kSlots];
    __shared__ uint32_t tmem_base;
    __shared__ int32_t rows[128];
    uint8_t *stages = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *slots = stages + S::kStages * S::kStageBytes;
    uint8_t *region = stages + S::kRoom;  // inner values in 32 bits, then their terms
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    if (t == 0) {
        for (int i = 0; i < S::kStages; ++i) {
            ptx::mbar_init(full + i, 1);
            ptx::mbar_init(empty + i, 1);
        }
        for (int i = 0; i < S::kStagesX; ++i) {
            ptx::mbar_init(full_x + i, 1);
            ptx::mbar_init(empty_x + i, 1);
        }
        for (int i = 0; i < 3; ++i) ptx::mbar_init(joined + i, 4 * S::kHalves * g.split);
        ptx::mbar_init(&inner_full, 1);
        ptx::mbar_init(&inner_ready, 4 * S::kHalves);
        for (int i = 0; i < kGroups; ++i) {
            ptx::mbar_init(sums_full + i, 1);
            ptx::mbar_init(sums_empty + i, 4);
        }
        for (int i = 0; i < S::kSlots; ++i) {
            ptx::mbar_init(base_full + i, 1);
            ptx::mbar_init(base_empty + i, 4);
        }
        ptx::mbar_init(&drained, 1);
        ptx::fence_barrier_init();
        ptx::prefetch_tensormap(&map_a);
        ptx::prefetch_tensormap(&map_b);
    }
    if (warp == 1) ptx::tmem_alloc(&tmem_base, 512);
    ptx::tc_fence_before();
    __syncthreads();
    if (g.split > 1) ptx::cluster_sync();  // the others' barriers are ready
    ptx::tc_fence_after();
    const uint32_t tmem = tmem_base;
    // After the tensor memory is taken, as in the product.  Beside k_adapters_few, the launch just before this one, this
    // kernel starts when every block of that one has waited for what was before both (or has gone, having waited): that is
    // complete, and its writes are in L2, where this kernel's reads go, by TMA or past L1.  The two write different rows
    // and read none of one another's; that one is waited for at the end, so that whoever waits for this one has both.
    ptx::launch_dependents();
    if (!g.beside) ptx::wait_dependencies();

    const int64_t tile = blockIdx.x / unsigned(g.split);
    const int rank = int(blockIdx.x % unsigned(g.split));
    int4 at = make_int4(0, 0, 0, 0);
    const bool mine = plan_tile(g.plan, g.tokens, g.adapters, g.which, tile, &at);
    const int count = at.z;
    const int64_t columns = (g.n + kColumns - 1) / kColumns;  // tiles of them
    const int64_t first_tile = columns * rank / g.split, last_tile = columns * (rank + 1) / g.split;
    [[maybe_unused]] const dbg::Side sb = dbg::side(g.base, 1, g.tokens, g.n, g.ld_base, 0, sizeof(T));
    [[maybe_unused]] const dbg::Side so = dbg::side(g.out, 1, g.tokens, g.n, g.ld_out, 0, sizeof(T));
    if (t < count) rows[t] = __ldcg(g.plan + plan_order_at(g.tokens, g.adapters) + at.y + t);
    __syncthreads();
    bool ok = true;

    if (!mine || at.x >= g.adapters || g.chunks == 0) {
        const int64_t j1 = last_tile * kColumns;
        if (mine && g.base != g.out) copy_rows<T>(g, rows, count, first_tile * kColumns, j1 < g.n ? j1 : g.n, !EDGE, sb, so);
    } else {
        const int first = int(int64_t(g.chunks) * rank / g.split), chunks = int(int64_t(g.chunks) * (rank + 1) / g.split) - first;
        const int tiles = int(last_tile - first_tile);
        // A tile's tokens that all lie side by side are one box, else 32 at a time are, else they go four rows to a load (the
        // last one's row fills up).  30 prompts of 8 adapters in turn, 8192 tokens, 8192 x 8192 rank 64: 246 us without boxes
        // of 32, 158 with them and nothing else (and one prompt to an adapter 76 us with a tile's box, 85 in boxes of 32).
        const bool together = rows[count - 1] - rows[0] == count - 1;
        uint32_t boxes = 0, rows_bytes = kTileX;  // of the warps that load
        if (!together && (warp == 0 || warp == 2)) {
            rows_bytes = 0;
            for (int r = 0; r < count; r += kBox) {
                const int last = (r + kBox < count ? r + kBox : count) - 1;
                const bool box = rows[last] - rows[r] == last - r;
                if (box) boxes |= 1u << (r / kBox);
                rows_bytes += box ? kBox * 128 : (last - r + 4) / 4 * 512;
            }
        }
        auto load_rows = [&](uint8_t *dst, const CUtensorMap *all, const CUtensorMap *box, const CUtensorMap *four, uint64_t *bar, int32_t c) {
            if (together) {
                ptx::tma_load_2d(dst, all, bar, c, rows[0]);
                return;
            }
            for (int r0 = 0; r0 < count; r0 += kBox) {
                if (boxes >> (r0 / kBox) & 1) {
                    ptx::tma_load_2d(dst + r0 * 128, box, bar, c, rows[r0]);
                    continue;
                }
                const int last = (r0 + kBox < count ? r0 + kBox : count) - 1;
                for (int r = r0; r <= last; r += 4)
                    ptx::tma_gather4(dst + r * 128, four, bar, c, rows[r], rows[r + 1 < last ? r + 1 : last],
                                     rows[r + 2 < last ? r + 2 : last], rows[r + 3 < last ? r + 3 : last]);
            }
        };
        constexpr int kPiece = 128 / int(sizeof(T)), kPieces = kColumns / kPiece;  // columns of a piece of base; pieces of a tile
        if (warp == 0) {
            // The whole warp waits and one elected lane issues, here and below: the 30 prompts above took 118 us (116 now),
            // 137 with these copies inside `lane == 0`, 131 with those of base there.
            const bool leader = ptx::elect_one();
            int c = 0, i = 0;
            for (; c < chunks; ++c) {
                const int s = c % S::kStagesX;
                if (c >= S::kStagesX) ok = ptx::mbar_wait_bounded(empty_x + s, (c / S::kStagesX - 1) & 1);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                uint8_t *dst = stages + s * S::kStageBytes;
                const int32_t k0 = (first + c) * 64;
                if (leader) {
                    ptx::mbar_arrive_expect_tx(full_x + s, RP * 128 + rows_bytes);
                    ptx::tma_load_3d(dst + kTileX, &map_a, full_x + s, k0, 0, at.x);
                    load_rows(dst, &map_x, &map_x32, &map_rows, full_x + s, k0);
                }
            }
            // Nothing may arrive after the block has gone, nor into memory that is used for something else.
            if (!leave_ring<S::kStagesX>(
                    c, [&](int s, uint32_t parity) { return ptx::mbar_wait_bounded(empty_x + s, parity); },
                    [&](int s, uint32_t parity) { ptx::mbar_wait_bounded(full_x + s, parity); }))
                ok = false;
            ok = __all_sync(0xffffffffu, ok);
            for (; i < tiles && ok; ++i) {
                const int s = i % S::kStages;
                if (i >= S::kStages) ok = ptx::mbar_wait_bounded(empty + s, (i / S::kStages - 1) & 1);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                if (leader) {
                    ptx::mbar_arrive_expect_tx(full + s, (RP + 63) / 64 * kTileX);
                    for (int k = 0; k < RP; k += 64)
                        ptx::tma_load_3d(stages + s * S::kStageBytes + k / 64 * kTileX, &map_b, full + s, k, int32_t((first_tile + i) * kColumns), at.x);
                }
            }
            if (!leave_ring<S::kStages>(
                    i, [&](int s, uint32_t parity) { return ptx::mbar_wait_bounded(empty + s, parity); },
                    [&](int s, uint32_t parity) { ptx::mbar_wait_bounded(full + s, parity); }))
                ok = false;
        } else if (warp == 1) {
            const bool leader = ptx::elect_one();
            const uint32_t idesc_a = ptx::bf16_idesc(128, RP), idesc_b = ptx::bf16_idesc(128, kColumns);
            for (int c = 0; c < chunks && ok; ++c) {
                const int s = c % S::kStagesX;
                ok = ptx::mbar_wait_bounded(full_x + s, (c / S::kStagesX) & 1);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                ptx::tc_fence_after();
                const uint32_t p = ptx::smem_addr(stages + s * S::kStageBytes);
                const uint64_t dx = ptx::operand_desc(p), da = ptx::operand_desc(p + kTileX);
                if (leader) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) ptx::mma_bf16(tmem, dx + 2 * k, da + 2 * k, idesc_a, c > 0 || k > 0);
                    ptx::mma_commit(empty_x + s);
                    if (c + 1 == chunks) ptx::mma_commit(&inner_full);
                }
            }
            __syncwarp();
            ok = ok && ptx::mbar_wait_bounded(&inner_ready, 0);
            const uint32_t v = ptx::smem_addr(region + S::kTermsAt);
            for (int i = 0; i < tiles && ok; ++i) {
                const int s = i % S::kStages, b = i % kGroups;
                ok = ok && ptx::mbar_wait_bounded(full + s, (i / S::kStages) & 1) &&
                     (i < kGroups || ptx::mbar_wait_bounded(sums_empty + b, (i / kGroups - 1) & 1));
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                ptx::tc_fence_after();
                const uint32_t p = ptx::smem_addr(stages + s * S::kStageBytes);
                if (leader) {
#pragma unroll
                    for (int k = 0; k < TERMS * RP; k += 16) {
                        const int kb = k % RP;
                        ptx::mma_bf16(tmem + b * kColumns, ptx::operand_desc(v + k / 64 * kTileX) + 2 * (k % 64 / 16),
                                      ptx::operand_desc(p + kb / 64 * kTileX) + 2 * (kb % 64 / 16), idesc_b, k > 0);
                    }
                    ptx::mma_commit(sums_full + b);
                    ptx::mma_commit(empty + s);
                }
            }
            if (!ok) {
                if (leader) ptx::mma_commit(&drained);
                ptx::mbar_wait_bounded(&drained, 0);
            }
        } else if (warp < 4) {
            const bool leader = ptx::elect_one();
            const int pieces = EDGE || warp != 2 ? 0 : tiles * kPieces;
            if (pieces && chunks) ok = ptx::mbar_wait_bounded(&inner_full, 0);  // the slots were stages
            for (int p = 0; p < pieces; ++p) {
                const int i = p / kPieces, mine = i / kGroups * kPieces + p % kPieces;  // of the group's pieces
                const int slot = i % kGroups * S::kPer + mine % S::kPer;
                if (ok && mine >= S::kPer) ok = ptx::mbar_wait_bounded(base_empty + slot, (mine / S::kPer - 1) & 1);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                if (!leader) continue;
                if (!g.base) {
                    ptx::mbar_arrive(base_full + slot);
                    continue;
                }
                ptx::mbar_arrive_expect_tx(base_full + slot, rows_bytes);
                load_rows(slots + slot * kTileX, &map_base, &map_base32, &map_base_rows, base_full + slot, int32_t(first_tile) * kColumns + p * kPiece);
            }
            if (!ok)  // no load may land after the block has gone
                for (int i = 0; i < S::kSlots; ++i) {
                    ptx::mbar_wait_bounded(base_full + i, 0, 10000000);
                    ptx::mbar_wait_bounded(base_full + i, 1, 10000000);
                }
        } else {
            const int w = warp & 3;  // the quarter of the lanes this warp may read
            const int row = w * 32 + lane, th = t - 128, group = (warp - 4) / 4;
            const uint32_t lanes = uint32_t(w * 32) << 16;
            const int n = int(g.n), j_first = int(first_tile) * kColumns, left = count - w * 32;  // rows of this warp
            // EDGE: a lane's column of base in each of the warp's rows, whose places the lanes hold.  Where there is no
            // such row or column, the first row's last column: loads without a branch or a predicate to set up.
            const int64_t own_token = EDGE && left > 0 ? rows[w * 32 + (lane < left ? lane : 0)] : 0;
            const int64_t own_base = own_token * g.ld_base, own_out = own_token * g.ld_out;
            auto old_value = [&](int r, int j) {
                const T *p = static_cast<const T *>(g.base) + __shfl_sync(0xffffffffu, own_base, r) + (j < n ? j : n - 1);
                return g.base && left > 0 && TR_LOAD_OK(sb, p, int(sizeof(T))) ? __ldcg(p) : T(0.0f);
            };
            [[maybe_unused]] T old[EDGE ? 32 : 1];
            if constexpr (EDGE) {
#pragma unroll
                for (int r = 0; r < 32; ++r) old[r] = old_value(r, j_first + group * kColumns + lane);
            }
            if (group < S::kHalves) {
                const float scale = g.scale ? __ldcg(g.scale + at.x) : 1.0f;
                constexpr int W = RP / S::kHalves;  // inner values to a thread
                const int c0 = group * W;
                float v[W];
                // Inner values of this lane's token, from this CTA's part of k.
                if (chunks) {
                    if (ok) ok = ptx::mbar_wait_bounded(&inner_full, 0);
                    __syncwarp();
                    ptx::tc_fence_after();
                    if constexpr (W == 16) {
                        ptx::tmem_load16(v, tmem + lanes + c0);
                        ptx::tmem_wait_load16(v);
                    } else {
#pragma unroll
                        for (int c = 0; c < W; c += 32) {
                            float part[32];
                            ptx::tmem_load32(part, tmem + lanes + c0 + c);
                            ptx::tmem_wait_load32(part);
#pragma unroll
                            for (int k = 0; k < 32; ++k) v[c + k] = part[k];
                        }
                    }
                    ptx::tc_fence_before();
                } else {
#pragma unroll
                    for (int c = 0; c < W; ++c) v[c] = 0.0f;
                }
                if (g.split > 1) {
                    float *inner = reinterpret_cast<float *>(region);
#pragma unroll
                    for (int c = 0; c < W; c += 4)
                        *reinterpret_cast<float4 *>(inner + inner_at<RP>(row, c0 + c)) = make_float4(v[c], v[c + 1], v[c + 2], v[c + 3]);
                    // A warp tells every CTA that it has come to a point, and waits until all warps have.
                    auto meet = [&](int k) {
                        __syncwarp();
                        if (lane < g.split) ptx::mbar_arrive_release_at(ptx::peer_addr(joined + k, uint32_t(lane)));
                        if (ok) ok = ptx::mbar_wait_cluster(joined + k, 0);
                        __syncwarp();
                    };
                    meet(0);
                    if (g.split == 2) {
                        // Both parts of the row, in rank order.
                        const uint32_t one = ptx::peer_addr(inner, 0), two = ptx::peer_addr(inner, 1);
#pragma unroll
                        for (int c = 0; c < W; c += 4) {
                            const int word = 4 * inner_at<RP>(row, c0 + c);
                            const float4 a = ptx::load_cluster4(one + word), b = ptx::load_cluster4(two + word);
                            v[c] = a.x + b.x;
                            v[c + 1] = a.y + b.y;
                            v[c + 2] = a.z + b.z;
                            v[c + 3] = a.w + b.w;
                        }
                    } else {
                        // Join the parts of 128 / split tokens, in rank order, in their place here: nobody else reads it.
                        const int share = 128 / g.split;
                        for (int k = th; k < share * (RP / 4); k += 128 * S::kHalves) {
                            const int r = rank * share + k / (RP / 4), c = k % (RP / 4) * 4;
                            if (r >= count) continue;
                            float *p = inner + inner_at<RP>(r, c);
                            float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                            float4 f[8];  // all on their way before the first is used
#pragma unroll
                            for (int peer = 0; peer < 8; ++peer)
                                if (peer < g.split) f[peer] = ptx::load_cluster4(ptx::peer_addr(p, uint32_t(peer)));
#pragma unroll
                            for (int peer = 0; peer < 8; ++peer)
                                if (peer < g.split) sum = make_float4(sum.x + f[peer].x, sum.y + f[peer].y, sum.z + f[peer].z, sum.w + f[peer].w);
                            *reinterpret_cast<float4 *>(p) = sum;
                        }
                        meet(1);
                        if (row < count) {
                            const uint32_t from = ptx::peer_addr(inner, uint32_t(row / share));
#pragma unroll
                            for (int c = 0; c < W; c += 4) {
                                const float4 f = ptx::load_cluster4(from + 4 * inner_at<RP>(row, c0 + c));
                                v[c] = f.x;
                                v[c + 1] = f.y;
                                v[c + 2] = f.z;
                                v[c + 3] = f.w;
                            }
                        }
                    }
                    if constexpr (!S::kApart) meet(2);  // every CTA has what it needs of the others: the region is free
                }
                // The terms of the inner values, 8 to a 16-byte chunk of a row in the 128-byte swizzle.
#pragma unroll
                for (int c = 0; c < W; c += 8) {
                    uint32_t word[4][TERMS];
#pragma unroll
                    for (int k = 0; k < 8; k += 2)
                        terms_of<TERMS>(c0 + c + k < g.rank ? __fmul_rn(v[c + k], scale) : 0.0f,  // rounded, whatever is taken from it
                                        c0 + c + k + 1 < g.rank ? __fmul_rn(v[c + k + 1], scale) : 0.0f, word[k / 2]);
#pragma unroll
                    for (int term = 0; term < TERMS; ++term) {
                        const int col = term * RP + c0 + c;
                        *reinterpret_cast<uint4 *>(region + S::kTermsAt + col / 64 * kTileX + row * 128 + ((col % 64 * 2) ^ ((row & 7) << 4))) =
                            make_uint4(word[0][term], word[1][term], word[2][term], word[3][term]);
                    }
                }
                ptx::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&inner_ready);
            }
            for (int i = group; i < tiles; i += kGroups) {
                if (ok) ok = ptx::mbar_wait_bounded(sums_full + group, (i / kGroups) & 1);
                __syncwarp();
                ptx::tc_fence_after();
                const uint32_t from = tmem + lanes + group * kColumns;
                if constexpr (!EDGE) {
                    constexpr int V = 16 / int(sizeof(T));
#pragma unroll
                    for (int p = 0; p < kPieces; ++p) {
                        const int mine = i / kGroups * kPieces + p, slot = group * S::kPer + mine % S::kPer;
                        if (ok) ok = ptx::mbar_wait_bounded(base_full + slot, (mine / S::kPer) & 1);
                        __syncwarp();
                        if (left > 0) {
                            // Every step's accesses are under way before the first is used.
                            const uint32_t piece = ptx::smem_addr(slots + slot * kTileX), own = piece + row * 128;
#pragma unroll
                            for (int c = 0; c < kPiece; c += 32) {
                                uint4 old[32 / V];
#pragma unroll
                                for (int k = 0; k < 32 / V; ++k)
                                    old[k] = g.base ? ptx::load_shared_16(own + (((c / V + k) ^ (row & 7)) << 4)) : make_uint4(0u, 0u, 0u, 0u);
                                float sums[32];
                                ptx::tmem_load32(sums, from + p * kPiece + c);
                                ptx::tmem_wait_load32(sums);
#pragma unroll
                                for (int k = 0; k < 32; k += V) {
                                    const int at = (c + k) / V;
                                    const Pack<T, V> b = *reinterpret_cast<const Pack<T, V> *>(&old[k / V]);
                                    float f[V];
#pragma unroll
                                    for (int q = 0; q < V; ++q) f[q] = sums[k + q] + b.get(q);
                                    Pack<T, V> o;
                                    o.round(f);
                                    ptx::store_shared_16(own + ((at ^ (row & 7)) << 4), *reinterpret_cast<const uint4 *>(&o));
                                }
                            }
                            __syncwarp();
                            const int j = j_first + i * kColumns + p * kPiece + lane % 8 * V;
                            uint4 was[8];
                            int32_t token[8];  // read here: registers are short while the sums are there
#pragma unroll
                            for (int l = 0; l < 8; ++l) {
                                const int r = l * 4 + lane / 8;
                                token[l] = rows[w * 32 + r];
                                was[l] = ptx::load_shared_16(piece + (w * 32 + r) * 128 + ((lane ^ r) % 8 << 4));
                            }
#pragma unroll
                            for (int l = 0; l < 8; ++l)
                                if (l * 4 + lane / 8 < left && j < n) {
                                    T *o = static_cast<T *>(g.out) + token[l] * g.ld_out + j;
                                    if (TR_STORE_OK(so, o, 16)) *reinterpret_cast<uint4 *>(o) = was[l];
                                }
                            ptx::fence_proxy_async_smem();
                        }
                        __syncwarp();
                        if (lane == 0) ptx::mbar_arrive(base_empty + slot);
                    }
                } else if (left > 0) {
                    // A quarter of the columns at a time goes through shared memory, so that lanes take neighbouring
                    // columns; base's values of the next quarter are on their way meanwhile.
                    uint4 *staging = reinterpret_cast<uint4 *>(slots) + (warp - 4) * 256;
#pragma unroll 1
                    for (int q = 0; q < 4; ++q) {
                        const int j = j_first + i * kColumns + q * 32 + lane;
                        const int j_next = q < 3 ? j + 32 : i + kGroups < tiles ? j + kGroups * kColumns - 96 : n;
                        float sums[32];
                        ptx::tmem_load32(sums, from + q * 32);
                        ptx::tmem_wait_load32(sums);
#pragma unroll
                        for (int c = 0; c < 8; ++c)
                            staging[lane * 8 + (c ^ (lane & 7))] = make_uint4(__float_as_uint(sums[4 * c]), __float_as_uint(sums[4 * c + 1]),
                                                                              __float_as_uint(sums[4 * c + 2]), __float_as_uint(sums[4 * c + 3]));
                        __syncwarp();
                        // base's values are used up before the next are asked for, and those before the stores: a wait
                        // for a value waits for all loads before it.
#pragma unroll
                        for (int r = 0; r < 32; ++r)
                            sums[r] = reinterpret_cast<const float *>(staging)[(r * 8 + ((lane >> 2) ^ (r & 7))) * 4 + (lane & 3)] + to_f32(old[r]);
#pragma unroll
                        for (int r = 0; r < 32; r += 8) {
#pragma unroll
                            for (int k = r; k < r + 8; ++k) old[k] = old_value(k, j_next);
#pragma unroll
                            for (int k = r; k < r + 8; ++k) {
                                T *o = static_cast<T *>(g.out) + __shfl_sync(0xffffffffu, own_out, k) + j;
                                if (k < left && j < n && TR_STORE_OK(so, o, int(sizeof(T)))) put_value(o, sums[k]);
                            }
                        }
                        __syncwarp();
                    }
                }
                ptx::tc_fence_before();  // the tensor cores may go on
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive_relaxed(sums_empty + group);
            }
        }
    }
    if (!ok) atomicOr(&g_fault_flag_adapters, kFaultWait);
    __syncwarp();
    ptx::tc_fence_before();
    __syncthreads();
    if (g.split > 1) ptx::cluster_sync();  // nobody leaves while another may read its shared memory, whatever ran out before
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_free(tmem, 512);
    }
    if (g.beside) ptx::wait_dependencies();
}

// --- a few tokens ---------------------------------------------------------------------------
//
// Next tokens of many requests: most adapters have a token or two, and what counts is how soon the adapters' bytes are
// here.  Tiles of up to 16 tokens, others 16 at a time.  A cluster to a tile as above, but no tensor memory, tensor maps or rings to set up: each warp reads its
// part of the adapter straight into the fragments of warp-wide matrix instructions, 16 tokens by 8 ranks (columns).
// The order of a contraction is free, so a lane's 16 contiguous bytes serve as the fragments of two
// instructions.  The columns of four instructions are spread so that a lane ends up with 8 neighbouring ones.

struct Few {
    const __nv_bfloat16 *x, *a, *b;
    const float *scale;
    const int32_t *plan;
    const void *base;
    void *out;
    int64_t tokens, adapters, ld_x, ld_a, stride_a, ld_b, stride_b, ld_base, ld_out;
    int32_t rank, k, n, split, which;
};

// Up to kFewTokens tokens (kFewTokensNarrow with ranks up to 16) this kernel works alone, up to kBothTokens on the small
// tiles.  What decides, tokens to an adapter, only the device knows; each limit buys one kind of batch with another.
// 8192 x 8192 bf16, one set of adapters again and again, us, alone and both:
//   rank 16   64 tokens of 48 adapters 13.2 and 13.8, of one 22.2 and 19.2; 128 of 48 13.3 and 14.6, of one 42 and 21; alone
//             is a launch and six tensor maps less for the host
//   rank 32   48 tokens of 48 adapters 17.0 and 17.7, of one 22.1 and 20.3; 64 of one 28.5 and 20.5
// Both, and k_adapters alone (a next token then takes a tile of 128):
//   rank 16   8 prompts 23.6 and 22.0 (1024 tokens), 35 and 34 (2048), 75 and 74 (8192); with 48 next tokens 35 and 48,
//             57 and 54, 121 and 102
//   rank 64   8 prompts 29.6 and 27.3, 43 and 40, 82 and 80; with 48 next tokens 52 and 56, 72 and 65, 153 and 114
constexpr int64_t kFewTokens = 32, kFewTokensNarrow = 64, kBothTokens = 2048;
constexpr int kFewThreads = 256, kFewWarps = kFewThreads / 32;

// D[16][8] += A[16][16] B[8][16]^T, a fragment's words being pairs along the contraction.
__device__ __forceinline__ void mma_16x8(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// N (4 or 8) values of a row from column c on, zeros from `cols` on and where there is no row.  WHOLE: all of them
// are below `cols` or none is; a load without a branch, so that many can be under way.
template <int N, bool WHOLE>
__device__ __forceinline__ uint4 values(const __nv_bfloat16 *row, int c, int cols, bool have, const dbg::Side &s) {
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if constexpr (WHOLE) {
        if (have && c < cols && TR_LOAD_OK(s, row + c, 2 * N)) {
            if constexpr (N == 8) {
                v = *reinterpret_cast<const uint4 *>(row + c);
            } else {
                const uint2 two = *reinterpret_cast<const uint2 *>(row + c);
                v.x = two.x;
                v.y = two.y;
            }
        }
        return v;
    }
    if (!have) return v;
    uint32_t w[4] = {};
#pragma unroll
    for (int q = 0; q < N; ++q)
        if (c + q < cols && TR_LOAD_OK(s, row + c + q, 2)) w[q / 2] |= uint32_t(__bfloat16_as_ushort(row[c + q])) << (q % 2 * 16);
    return make_uint4(w[0], w[1], w[2], w[3]);
}

constexpr int few_shares(int rp) { return rp <= 32 ? 1 : rp / 32; }

// EDGE: as above.
template <int RP, typename T, bool EDGE>
__global__ void __launch_bounds__(kFewThreads, 2) k_adapters_few(const Few g) {
    ptx::wait_dependencies();
    ptx::launch_dependents();  // in this order, in every block: k_adapters beside this one counts on it
    constexpr int TERMS = sizeof(T) == 2 ? 2 : 3;
    constexpr int RC = RP == 16 ? 4 : 8, STEPS = RP / (4 * RC);  // values of a row of b to a lane and step
    constexpr int PITCH = RP + 8;                                // of the terms, in values
    constexpr int AHEAD = RP <= 64 ? 2 : 1;                      // units of 32 columns whose b and base are read before the inner values are there
    constexpr int SHARES = few_shares(RP), RW = RP / SHARES;     // warps share the ranks first, RW to each, then k
    extern __shared__ float part[];                              // [warps / SHARES][16][RP]
    __shared__ float sums[16][RP + 4];
    __shared__ alignas(16) __nv_bfloat16 terms[TERMS][16][PITCH];
    __shared__ int32_t rows[128];
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5, gid = lane >> 2, tid = lane & 3;
    const int64_t tile = blockIdx.x / unsigned(g.split);
    const int rank = int(blockIdx.x % unsigned(g.split));
    int4 at;
    if (!plan_tile(g.plan, g.tokens, g.adapters, g.which, tile, &at)) return;  // the whole cluster
    const int count = at.z;
    if (t < count) rows[t] = g.plan[plan_order_at(g.tokens, g.adapters) + at.y + t];
    __syncthreads();
    [[maybe_unused]] const dbg::Side sx = dbg::side(g.x, 1, g.tokens, g.k, g.ld_x, 0, 2);
    [[maybe_unused]] const dbg::Side sa = dbg::side(g.a, g.adapters, g.rank, g.k, g.ld_a, g.stride_a, 2);
    [[maybe_unused]] const dbg::Side sv = dbg::side(g.b, g.adapters, g.n, g.rank, g.ld_b, g.stride_b, 2);
    [[maybe_unused]] const dbg::Side sb = dbg::side(g.base, 1, g.tokens, g.n, g.ld_base, 0, sizeof(T));
    [[maybe_unused]] const dbg::Side so = dbg::side(g.out, 1, g.tokens, g.n, g.ld_out, 0, sizeof(T));
    const int units = (g.n + 31) / 32, first = int(int64_t(units) * rank / g.split), last = int(int64_t(units) * (rank + 1) / g.split);
    const bool bare = at.x >= g.adapters || g.k == 0;
    if (bare && g.base == g.out) return;
    const int runs = (g.k + 31) / 32;  // of 32 values of k
    const int run0 = int(int64_t(runs) * rank / g.split), run1 = int(int64_t(runs) * (rank + 1) / g.split);
    const __nv_bfloat16 *a = g.a + at.x * g.stride_a, *b = g.b + at.x * g.stride_b;
    const float scale = bare ? 0.0f : g.scale ? g.scale[at.x] : 1.0f;
    // What b's loads will find in L2 when the inner values are there.
    if (!bare) {
        constexpr int ROWS = 64 / RP ? 64 / RP : 1;  // of b to 128 bytes, about
        for (int col = first * 32 + t * ROWS; col < last * 32 && col < g.n; col += kFewThreads * ROWS)
            for (int r = 0; r < g.rank; r += 64) ptx::prefetch_l2(b + col * g.ld_b + r);
    }

    for (int m0 = 0; m0 < count; m0 += 16) {
        // The two tokens of this lane's rows of a fragment.
        const bool has[2] = {m0 + gid < count, m0 + gid + 8 < count};
        const int64_t token[2] = {has[0] ? rows[m0 + gid] : 0, has[1] ? rows[m0 + gid + 8] : 0};
        if (!bare) {
            float acc[RW / 8][4] = {};
            const __nv_bfloat16 *x0 = g.x + token[0] * g.ld_x, *x1 = g.x + token[1] * g.ld_x;
            const int r0 = warp % SHARES * RW, depth = warp / SHARES;
            auto add = [&](int run, auto whole) {
                constexpr bool W = decltype(whole)::value;
                const int c = run * 32 + tid * 8;
                const uint4 u = values<8, W>(x0, c, g.k, has[0], sx), v = values<8, W>(x1, c, g.k, has[1], sx);
                uint4 w[RW / 8];
#pragma unroll
                for (int j = 0; j < RW / 8; ++j) {
                    const int r = r0 + j * 8 + gid;
                    w[j] = values<8, W>(a + r * g.ld_a, c, g.k, r < g.rank, sa);
                }
#pragma unroll
                for (int j = 0; j < RW / 8; ++j) {
                    mma_16x8(acc[j], u.x, v.x, u.y, v.y, w[j].x, w[j].y);
                    mma_16x8(acc[j], u.z, v.z, u.w, v.w, w[j].z, w[j].w);
                }
            };
            const bool ragged = g.k % 8 != 0 && run1 == runs;  // the last run is of pieces
            constexpr int EACH = kFewWarps / SHARES;           // warps along k
            int run = run0 + depth;
            const int end = ragged ? run1 - 1 : run1;
            for (; run + 3 * EACH < end; run += 4 * EACH) {
#pragma unroll
                for (int q = 0; q < 4; ++q) add(run + q * EACH, std::true_type());
            }
            for (; run < end; run += EACH) add(run, std::true_type());
            if (run < run1) add(run, std::false_type());
#pragma unroll
            for (int j = 0; j < RW / 8; ++j) {
                float *p = part + (depth * 16 + gid) * RP + r0 + j * 8 + tid * 2;
                *reinterpret_cast<float2 *>(p) = make_float2(acc[j][0], acc[j][1]);
                *reinterpret_cast<float2 *>(p + 8 * RP) = make_float2(acc[j][2], acc[j][3]);
            }
        }
        // Unit u: b's rows of its 32 columns and the lane's 8 columns of base.
        struct Unit {
            uint4 b[STEPS][4];
            Pack<T, 16 / int(sizeof(T))> base[2][sizeof(T) / 2];
        };
        constexpr int V = 16 / int(sizeof(T));
        const bool pieces = g.rank % RC != 0;
        auto read = [&](Unit &m, int u) {
            const bool here = u < last;
#pragma unroll
            for (int s = 0; s < STEPS; ++s)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int col = u * 32 + 8 * (gid >> 1) + 2 * j + (gid & 1);
                    const bool have = here && !bare && col < g.n;
                    m.b[s][j] = pieces ? values<RC, false>(b + col * g.ld_b, s * 4 * RC + tid * RC, g.rank, have, sv)
                                       : values<RC, true>(b + col * g.ld_b, s * 4 * RC + tid * RC, g.rank, have, sv);
                }
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int h = 0; h < int(sizeof(T)) / 2; ++h) {
                    m.base[r][h].clear();
                    const int col = u * 32 + 8 * tid + h * V;
                    const T *p = static_cast<const T *>(g.base) + token[r] * g.ld_base + col;
                    if (!g.base || !here || !has[r]) continue;
                    if constexpr (EDGE) {
#pragma unroll
                        for (int q = 0; q < V; ++q)
                            if (col + q < g.n && TR_LOAD_OK(sb, p + q, int(sizeof(T)))) m.base[r][h].set(q, p[q]);
                    } else {
                        if (col < g.n && TR_LOAD_OK(sb, p, 16)) m.base[r][h] = *reinterpret_cast<const Pack<T, V> *>(p);
                    }
                }
        };
        Unit unit[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) read(unit[i], first + warp + i * kFewWarps);
        if (!bare) {
            // The warps' parts, then the CTAs', both in order.
            __syncthreads();
            for (int i = t; i < 16 * RP; i += kFewThreads) {
                float v = 0.0f;
#pragma unroll
                for (int w = 0; w < kFewWarps / SHARES; ++w) v += part[w * 16 * RP + i];
                sums[i / RP][i % RP] = v;
            }
            if (g.split > 1) ptx::cluster_sync();
            else __syncthreads();
            for (int i = t; i < 16 * RP; i += kFewThreads) {
                const int m = i / RP, r = i % RP;
                float v = 0.0f, f[8];
#pragma unroll
                for (int peer = 0; peer < 8; ++peer)
                    if (peer < g.split) f[peer] = ptx::load_cluster(ptx::peer_addr(&sums[m][r], uint32_t(peer)));
#pragma unroll
                for (int peer = 0; peer < 8; ++peer)
                    if (peer < g.split) v += f[peer];
                uint32_t word[TERMS];
                terms_of<TERMS>(r < g.rank ? __fmul_rn(v, scale) : 0.0f, 0.0f, word);
#pragma unroll
                for (int term = 0; term < TERMS; ++term) terms[term][m][r] = __ushort_as_bfloat16(uint16_t(word[term]));
            }
            __syncthreads();
            if (g.split > 1) ptx::cluster_arrive();
        }
        auto finish = [&](const Unit &m, int u) {
            float d[4][4] = {};
            if (!bare)
#pragma unroll
                for (int term = 0; term < TERMS; ++term)
#pragma unroll
                    for (int s = 0; s < STEPS; ++s) {
                        const __nv_bfloat16 *p = &terms[term][gid][s * 4 * RC + tid * RC], *q = p + 8 * PITCH;
                        if constexpr (RC == 4) {
                            const uint2 v0 = *reinterpret_cast<const uint2 *>(p), v1 = *reinterpret_cast<const uint2 *>(q);
#pragma unroll
                            for (int j = 0; j < 4; ++j) mma_16x8(d[j], v0.x, v1.x, v0.y, v1.y, m.b[s][j].x, m.b[s][j].y);
                        } else {
                            const uint4 v0 = *reinterpret_cast<const uint4 *>(p), v1 = *reinterpret_cast<const uint4 *>(q);
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                mma_16x8(d[j], v0.x, v1.x, v0.y, v1.y, m.b[s][j].x, m.b[s][j].y);
                                mma_16x8(d[j], v0.z, v1.z, v0.w, v1.w, m.b[s][j].z, m.b[s][j].w);
                            }
                        }
                    }
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int h = 0; h < int(sizeof(T)) / 2; ++h) {
                    const int col = u * 32 + 8 * tid + h * V;
                    if (!has[r] || col >= g.n) continue;
                    float f[V];
#pragma unroll
                    for (int q = 0; q < V; ++q) f[q] = d[(h * V + q) / 2][2 * r + q % 2] + m.base[r][h].get(q);
                    Pack<T, V> o;
                    o.round(f);
                    T *p = static_cast<T *>(g.out) + token[r] * g.ld_out + col;
                    if constexpr (EDGE) {
#pragma unroll
                        for (int q = 0; q < V; ++q)
                            if (col + q < g.n && TR_STORE_OK(so, p + q, int(sizeof(T)))) p[q] = pack_elem(o, q);
                    } else {
                        if (TR_STORE_OK(so, p, 16)) *reinterpret_cast<Pack<T, V> *>(p) = o;
                    }
                }
        };
        for (int u = first + warp; u < last; u += AHEAD * kFewWarps)
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                if (u + i * kFewWarps >= last) continue;
                finish(unit[i], u + i * kFewWarps);
                read(unit[i], u + (i + AHEAD) * kFewWarps);
            }
        __syncwarp();
        if (!bare && g.split > 1) ptx::cluster_wait();  // nobody writes its sums anew, or leaves, before all have read them
    }
}

// Planes of rows x cols values of 2 or 4 bytes, or a matrix (planes 0): boxes of 128 bytes x box_rows.
bool encode(CUtensorMap *map, const void *base, int es, int64_t planes, int64_t rows, int64_t cols, int64_t ld, int64_t stride,
            int box_rows) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {cuuint64_t(cols), cuuint64_t(rows), cuuint64_t(planes)};
    const cuuint64_t strides[2] = {cuuint64_t(ld * es), cuuint64_t((planes > 1 ? stride : rows * ld) * es)};
    const cuuint32_t box[3] = {cuuint32_t(128 / es), cuuint32_t(box_rows), 1}, estr[3] = {1, 1, 1};
    return fn(map, es == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, planes ? 3 : 2, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A launch in clusters that may start while the kernel before it drains.
template <typename... K, typename... A>
cudaError_t launch_clusters(void (*kern)(K...), int64_t grid, int threads, size_t smem, int cluster, cudaStream_t stream, A &&...args) {
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
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, std::forward<A>(args)...);
    if (e != cudaSuccess) (void)cudaGetLastError();
    return e;
}

template <int RP, typename T, bool EDGE>
cudaError_t launch_few(Few g, int64_t tiles, cudaStream_t stream) {
    auto kern = k_adapters_few<RP, T, EDGE>;
    constexpr size_t smem = size_t(kFewWarps / few_shares(RP)) * 16 * RP * 4;
    // Eight CTAs to a tile, fewer where as many tiles as there can be would not be resident at one time, or a warp
    // would have less than a run of k and a unit of columns.
    const int64_t resident = 2 * int64_t(sm_count());
    g.split = 8;
    while (g.split > 1 && (tiles * g.split > resident || ((g.k + 31) / 32 < g.split * kFewWarps && (g.n + 31) / 32 < g.split * kFewWarps)))
        g.split /= 2;
    return launch_clusters(kern, tiles * g.split, kFewThreads, smem, g.split, stream, g);
}

template <int RP>
cudaError_t launch_few_rank(const Few &g, bool f32, bool edge, int64_t tiles, cudaStream_t stream) {
    if (f32) return edge ? launch_few<RP, float, true>(g, tiles, stream) : launch_few<RP, float, false>(g, tiles, stream);
    return edge ? launch_few<RP, __nv_bfloat16, true>(g, tiles, stream) : launch_few<RP, __nv_bfloat16, false>(g, tiles, stream);
}

template <int RP, typename T, bool EDGE>
cudaError_t launch_one(const CUtensorMap (&maps)[8], Adapt g, int64_t tiles, cudaStream_t stream) {
    using S = Shape<RP, sizeof(T) == 2 ? 2 : 3>;
    auto kern = k_adapters<RP, T, EDGE>;
    const cudaError_t e = allow_shared<k_adapters<RP, T, EDGE>>(S::kSmem);
    if (e != cudaSuccess) return e;
    // CTAs to a tile until the tiles fill what is resident at one time, each keeping two chunks of k or more.  How many
    // tiles there are is known on the device alone: the fewest that these tokens can make, and every second adapter's
    // end (2000 tokens of 8 adapters, 8192 x 8192: 25 tiles take 56 us with 8 CTAs to a tile, two waves).
    const int64_t resident = sm_count(), least = (g.tokens + kPlanTile - 1) / kPlanTile;
    const int64_t likely = least + (tiles < g.adapters + 1 ? tiles : g.adapters + 1) / 2;
    g.split = 1;
    while (g.split < 8 && likely * g.split * 2 <= resident && g.chunks >= g.split * 4) g.split *= 2;
    return launch_clusters(kern, tiles * g.split, kThreads, S::kSmem, g.split, stream, maps[0], maps[1], maps[2], maps[3], maps[4], maps[5], maps[6],
                           maps[7], g);
}

template <int RP>
cudaError_t launch_rank(const CUtensorMap (&maps)[8], const Adapt &g, bool f32, bool edge, int64_t tiles, cudaStream_t stream) {
    if (f32) return edge ? launch_one<RP, float, true>(maps, g, tiles, stream) : launch_one<RP, float, false>(maps, g, tiles, stream);
    return edge ? launch_one<RP, __nv_bfloat16, true>(maps, g, tiles, stream) : launch_one<RP, __nv_bfloat16, false>(maps, g, tiles, stream);
}

}  // namespace

TR_WAIT_UNIT(adapters)

// Debug builds: this unit's record of refused accesses.
TR_BOUNDS_READER(read_bounds_adapters)

cudaError_t launch_adapter_plan(const tr_adapter_plan_args &p) {
    const int64_t groups = p.adapters + 1;
    // As many warps as have counts in shared memory, and tokens.
    int64_t warps = (p.tokens + 31) / 32;
    const int64_t room = 200 * 1024 / (4 * groups);
    if (warps > room) warps = room;
    if (warps > kPlanThreads / 32) warps = kPlanThreads / 32;
    const cudaError_t e = allow_shared<k_adapter_plan>(200 * 1024);  // the most that any call needs
    if (e != cudaSuccess) return e;
    return launch_pdl(k_adapter_plan, dim3(1), dim3(kPlanThreads), size_t(warps * groups * 4), reinterpret_cast<cudaStream_t>(p.stream),
                      p.index, static_cast<int32_t *>(p.plan), int(p.tokens), int(p.adapters), int(warps));
}

cudaError_t launch_adapters(const tr_adapters_args &p, const char **why) {
    const bool f32 = p.out_dtype == TR_DTYPE_F32;
    const int es = f32 ? 4 : 2;
    const bool edge = (p.n * es) % 16 != 0 || !side_aligned16(p.out, p.ld_out, 0, 1, es) || (p.base && !side_aligned16(p.base, p.ld_base, 0, 1, es));
    const bool none = p.adapters == 0 || p.k == 0;  // nothing to add: base alone
    Adapt g{p.scale, static_cast<const int32_t *>(p.plan), p.base, p.out, p.tokens, p.adapters,
                  p.n, p.ld_base, p.ld_out, int32_t(p.rank), none ? 0 : int32_t((p.k + 63) / 64), 1, kAll, 0};
    const int rp = p.rank <= 16 ? 16 : p.rank <= 32 ? 32 : p.rank <= 64 ? 64 : 128;
    const int64_t tiles = plan_tiles(p.tokens, p.adapters);
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(p.stream);
    const bool alone = p.tokens <= (rp == 16 ? kFewTokensNarrow : kFewTokens);
    if (p.tokens <= kBothTokens) {
        const Few few{static_cast<const __nv_bfloat16 *>(p.x), static_cast<const __nv_bfloat16 *>(p.a), static_cast<const __nv_bfloat16 *>(p.b),
                      p.scale, g.plan, p.base, p.out, p.tokens, p.adapters, p.ld_x, p.ld_a, p.stride_a, p.ld_b, p.stride_b, p.ld_base, p.ld_out,
                      int32_t(p.rank), int32_t(none ? 0 : p.k), int32_t(p.n), 1, alone ? kAll : kSmall};
        // Each adapter, and those without one, has one small tile at the most.
        const int64_t small = alone || tiles < p.adapters + 1 ? tiles : p.adapters + 1;
        const cudaError_t e = rp == 16   ? launch_few_rank<16>(few, f32, edge, small, stream)
                              : rp == 32 ? launch_few_rank<32>(few, f32, edge, small, stream)
                              : rp == 64 ? launch_few_rank<64>(few, f32, edge, small, stream)
                                         : launch_few_rank<128>(few, f32, edge, small, stream);
        if (e != cudaSuccess || alone) return e;
        g.which = kLarge;
        g.beside = 1;  // nothing may be launched between the two
    }
    const int64_t large = g.beside ? plan_large_tiles(p.tokens, p.adapters) : tiles;
    CUtensorMap maps[8] = {};
    auto rows_maps = [&](CUtensorMap *m, const void *rows, int bytes, int64_t cols, int64_t ld) {
        return encode(m, rows, bytes, 0, p.tokens, cols, ld, 0, 128) && encode(m + 1, rows, bytes, 0, p.tokens, cols, ld, 0, kBox) &&
               encode(m + 2, rows, bytes, 0, p.tokens, cols, ld, 0, 1);
    };
    if (!none && (!rows_maps(maps, p.x, 2, p.k, p.ld_x) || !encode(maps + 3, p.a, 2, p.adapters, p.rank, p.k, p.ld_a, p.stride_a, rp) ||
                  !encode(maps + 4, p.b, 2, p.adapters, p.n, p.rank, p.ld_b, p.stride_b, kColumns) ||
                  (p.base && !edge && !rows_maps(maps + 5, p.base, es, p.n, p.ld_base)))) {
        *why = "adapters: cuTensorMapEncodeTiled rejected the operands (a pitch of 2^40 bytes or more)";
        return cudaErrorInvalidValue;
    }
    if (rp == 16) return launch_rank<16>(maps, g, f32, edge, large, stream);
    if (rp == 32) return launch_rank<32>(maps, g, f32, edge, large, stream);
    if (rp == 64) return launch_rank<64>(maps, g, f32, edge, large, stream);
    return launch_rank<128>(maps, g, f32, edge, large, stream);
}

}  // namespace tr

extern "C" int64_t tr_adapter_plan_bytes(int64_t tokens, int64_t adapters) {
    if (tokens < 0 || adapters < 0 || tokens >= int64_t(1) << 31 || adapters > tr::kMostAdapters) return -1;
    return tr::plan_bytes(tokens, adapters);
}

// Low-rank adapters of many requests at once: out[i] = base[i] + B_g (scale_g A_g x_i) for
// each token i with its own adapter g.
#include "adapter_plan.cuh"
#include "launch.cuh"
#include "row_chunk.cuh"
#include "tr_internal.h"

namespace tr {
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
    __shared__ int2 joined[32], carry;
    const int groups = adapters + 1, t = threadIdx.x, lane = t & 31, warp = t >> 5;
    [[maybe_unused]] const dbg::Side si = dbg::side(index, 1, 1, tokens, tokens, 0, 4);
    [[maybe_unused]] const dbg::Side sp = dbg::side(plan, 1, 1, plan_bytes(tokens, adapters) / 4, plan_bytes(tokens, adapters) / 4, 0, 4);
    for (int i = t; i < warps * groups; i += kPlanThreads) counts[i] = 0;
    if (t == 0) carry = make_int2(0, 0);
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
        for (int64_t i0 = first; i0 < last; i0 += 32) {
            const int64_t i = i0 + lane;
            const unsigned here = __ballot_sync(0xffffffffu, i < last);
            if (i < last) {
                const int g = group_of(i);
                const unsigned same = __match_any_sync(here, g);
                put(i, g, __popc(same & ((1u << lane) - 1)));
                __syncwarp(here);
                if (lane == 31 - __clz(same)) mine[g] += __popc(same);
            }
            __syncwarp();
        }
    };
    walk([](int64_t, int, int) {});
    __syncthreads();
    // Tokens before each adapter (x) and tiles before it (y), 1024 adapters at a time.
    for (int g0 = 0; g0 < groups; g0 += kPlanThreads) {
        const int g = g0 + t;
        int n = 0;
        if (g < groups)
            for (int w = 0; w < warps; ++w) n += counts[w * groups + g];
        const int2 own = make_int2(n, (n + kPlanTile - 1) / kPlanTile);
        int2 s = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, s.x, o), y = __shfl_up_sync(0xffffffffu, s.y, o);
            if (lane >= o) s = make_int2(s.x + x, s.y + y);
        }
        if (lane == 31) joined[warp] = s;
        __syncthreads();
        if (warp == 0) {
            int2 j = joined[lane];
            const int2 was = j;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, j.x, o), y = __shfl_up_sync(0xffffffffu, j.y, o);
                if (lane >= o) j = make_int2(j.x + x, j.y + y);
            }
            joined[lane] = make_int2(carry.x + j.x - was.x, carry.y + j.y - was.y);
            __syncwarp();
            if (lane == 31) carry = make_int2(carry.x + j.x, carry.y + j.y);
        }
        __syncthreads();
        if (g < groups) {
            int at = joined[warp].x + s.x - own.x;
            const int tile = joined[warp].y + s.y - own.y;
            for (int k = 0; k < own.y; ++k) {
                const int left = n - k * kPlanTile;
                int32_t *p = plan + plan_tiles_at() + 4 * int64_t(tile + k);
                if (TR_STORE_OK(sp, p, 16))
                    *reinterpret_cast<int4 *>(p) = make_int4(g, at + k * kPlanTile, left < kPlanTile ? left : kPlanTile, 0);
            }
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
    if (t == 0 && TR_STORE_OK(sp, plan, 16)) *reinterpret_cast<int4 *>(plan) = make_int4(carry.y, tokens, adapters, 0);
}

// --- the adapters ---------------------------------------------------------------------------

struct Adapt {
    const __nv_bfloat16 *x, *a, *b;
    const float *scale;
    const int32_t *plan;
    const void *base;
    void *out;
    int64_t tokens, adapters, k, n;
    int64_t ld_x, ld_a, stride_a, ld_b, stride_b, ld_base, ld_out;
    int rank;
};

// One token to a block.
template <typename T>
__global__ void __launch_bounds__(256) k_adapters_any(const Adapt a) {
    pdl_prologue();
    __shared__ float v[128];
    [[maybe_unused]] const dbg::Side sx = dbg::side(a.x, 1, a.tokens, a.k, a.ld_x, 0, 2);
    [[maybe_unused]] const dbg::Side sa = dbg::side(a.a, a.adapters, a.rank, a.k, a.ld_a, a.stride_a, 2);
    [[maybe_unused]] const dbg::Side sb = dbg::side(a.b, a.adapters, a.n, a.rank, a.ld_b, a.stride_b, 2);
    [[maybe_unused]] const dbg::Side ss = dbg::side(a.base, 1, a.tokens, a.n, a.ld_base, 0, sizeof(T));
    [[maybe_unused]] const dbg::Side so = dbg::side(a.out, 1, a.tokens, a.n, a.ld_out, 0, sizeof(T));
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (a.plan[1] != a.tokens || a.plan[2] != a.adapters) return;  // not these tokens' plan
    const int tiles = a.plan[0];
    const int32_t *order = a.plan + plan_order_at(a.tokens, a.adapters);
    for (int64_t at = blockIdx.x; at < int64_t(tiles) * kPlanTile; at += gridDim.x) {
        const int4 tile = *reinterpret_cast<const int4 *>(a.plan + plan_tiles_at() + 4 * (at / kPlanTile));
        if (at % kPlanTile >= tile.z) continue;
        const int64_t token = order[tile.y + at % kPlanTile], g = tile.x;
        const bool bare = g >= a.adapters;
        for (int r = warp; r < a.rank && !bare; r += 8) {
            const __nv_bfloat16 *x = a.x + token * a.ld_x, *row = a.a + g * a.stride_a + r * a.ld_a;
            float s = 0.0f;
            for (int64_t l = lane; l < a.k; l += 32)
                if (TR_LOAD_OK(sx, x + l, 2) && TR_LOAD_OK(sa, row + l, 2)) s = fmaf(to_f32(x[l]), to_f32(row[l]), s);
            s = warp_sum(s);
            if (lane == 0) v[r] = a.scale ? s * a.scale[g] : s;
        }
        __syncthreads();
        for (int64_t j = threadIdx.x; j < a.n; j += 256) {
            float s = 0.0f;
            const __nv_bfloat16 *row = a.b + g * a.stride_b + j * a.ld_b;
            for (int r = 0; r < a.rank && !bare; ++r)
                if (TR_LOAD_OK(sb, row + r, 2)) s = fmaf(v[r], to_f32(row[r]), s);
            const T *p = static_cast<const T *>(a.base) + token * a.ld_base + j;
            if (a.base && TR_LOAD_OK(ss, p, int(sizeof(T)))) s = bare ? to_f32(*p) : to_f32(*p) + s;
            T *o = static_cast<T *>(a.out) + token * a.ld_out + j;
            if (TR_STORE_OK(so, o, int(sizeof(T)))) put_value(o, s);
        }
        __syncthreads();
    }
}

}  // namespace

// Debug builds: this unit's record of refused accesses.
TR_BOUNDS_READER(read_bounds_adapters)

cudaError_t launch_adapter_plan(const tr_adapter_plan_args &p) {
    const int64_t groups = p.adapters + 1;
    // As many warps as have counts in shared memory, and tokens.
    int64_t warps = (p.tokens + 31) / 32;
    const int64_t room = 200 * 1024 / (4 * groups);
    if (warps > room) warps = room;
    if (warps > kPlanThreads / 32) warps = kPlanThreads / 32;
    // Always the most that any call needs: threads with other sizes set it too.
    const cudaError_t e = cudaFuncSetAttribute(k_adapter_plan, cudaFuncAttributeMaxDynamicSharedMemorySize, 200 * 1024);
    if (e != cudaSuccess) return e;
    return launch_pdl(k_adapter_plan, dim3(1), dim3(kPlanThreads), size_t(warps * groups * 4), reinterpret_cast<cudaStream_t>(p.stream),
                      p.index, static_cast<int32_t *>(p.plan), int(p.tokens), int(p.adapters), int(warps));
}

cudaError_t launch_adapters(const tr_adapters_args &p) {
    const Adapt a{static_cast<const __nv_bfloat16 *>(p.x), static_cast<const __nv_bfloat16 *>(p.a), static_cast<const __nv_bfloat16 *>(p.b),
                  p.scale, static_cast<const int32_t *>(p.plan), p.base, p.out, p.tokens, p.adapters, p.k, p.n,
                  p.ld_x, p.ld_a, p.stride_a, p.ld_b, p.stride_b, p.ld_base, p.ld_out, int(p.rank)};
    const int64_t most = int64_t(1) << 30, work = plan_tiles(p.tokens, p.adapters) * kPlanTile;
    const dim3 grid(unsigned(work < most ? work : most));
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(p.stream);
    return p.out_dtype == TR_DTYPE_F32 ? launch_pdl(k_adapters_any<float>, grid, dim3(256), 0, stream, a)
                                       : launch_pdl(k_adapters_any<__nv_bfloat16>, grid, dim3(256), 0, stream, a);
}

}  // namespace tr

extern "C" int64_t tr_adapter_plan_bytes(int64_t tokens, int64_t adapters) {
    if (tokens < 0 || adapters < 0 || tokens >= int64_t(1) << 31 || adapters > tr::kMostAdapters) return -1;
    return tr::plan_bytes(tokens, adapters);
}

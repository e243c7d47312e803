// The plan of a batch's adapters in memory: 32-bit words that k_adapter_plan writes and
// tr_adapters walks.  For the device and, for its size, the host.
#pragma once

#include <cstdint>

namespace tr {

constexpr int kPlanTile = 128;              // tokens of one adapter that are worked on together, at the most
constexpr int kPlanFew = 16;                // tokens of a small tile, at the most
constexpr int64_t kPlanHead = 4;            // large tiles, tokens, adapters, small tiles
constexpr int64_t kMostAdapters = 32767;    // a warp's counts of them fit shared memory

// Tiles of `tokens` tokens at the most: every adapter, and those without one, may end
// inside a tile.
__host__ __device__ inline int64_t plan_tiles(int64_t tokens, int64_t adapters) {
    const int64_t groups = tokens < adapters + 1 ? tokens : adapters + 1;
    return (tokens - groups) / kPlanTile + groups;
}

// Of those with more than kPlanFew tokens.
__host__ __device__ inline int64_t plan_large_tiles(int64_t tokens, int64_t adapters) {
    const int64_t most = tokens / (kPlanFew + 1), tiles = plan_tiles(tokens, adapters);
    return most < tiles ? most : tiles;
}

// Places, in words, of the tiles -- {adapter (adapters: none), place in the order, tokens, 0} each, the large ones from
// the front, the small ones from the back -- and of the order of the tokens.
__host__ __device__ inline int64_t plan_tiles_at() { return kPlanHead; }
__host__ __device__ inline int64_t plan_order_at(int64_t tokens, int64_t adapters) {
    return kPlanHead + 4 * plan_tiles(tokens, adapters);
}
__host__ __device__ inline int64_t plan_bytes(int64_t tokens, int64_t adapters) {
    return 4 * (plan_order_at(tokens, adapters) + tokens);
}

}  // namespace tr

// A ring of rows that bulk copies keep in flight: what the norms' kernels that walk many rows share.
#pragma once

#include <cstdint>

namespace tr {

constexpr int kMaxStages = 8;

// Shared memory that each of n blocks to an SM may ask for: 228 KB less what the
// system (1 KB) and the kernel's own words take of every block.
constexpr uint32_t ring_room(int64_t n) { return uint32_t(228 * 1024 / n) - 2048; }

// One row as a bulk copy takes it: the 16-byte granules that hold it.
struct Granules {
    const uint8_t *src;
    uint32_t shift, bytes;  // of the row's first byte past src; of the copy
    bool inside;            // every granule lies between the matrix's first and last value
};

template <typename T>
__device__ __forceinline__ Granules granules(const void *base, int64_t rows, int64_t cols, int64_t ld,
                                             int64_t row) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(base);
    const uintptr_t hi = lo + uintptr_t((rows - 1) * ld + cols) * sizeof(T);
    const uintptr_t a = lo + uintptr_t(row * ld) * sizeof(T), b = a + uintptr_t(cols) * sizeof(T);
    const uintptr_t first = a & ~uintptr_t(15), last = (b + 15) & ~uintptr_t(15);
    return Granules{reinterpret_cast<const uint8_t *>(first), uint32_t(a - first), uint32_t(last - first),
                    first >= lo && last <= hi};
}

}  // namespace tr

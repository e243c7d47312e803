// How the warpgroups of a block of k_matmul_pair share its registers.  Host code too:
// the launch checks it.
#pragma once

namespace tr {

constexpr int kPairThreads = 384;  // a warpgroup of loads and instructions, two that add
// Registers of a thread in the first warpgroup and in the other two: 56 x 128 + 224 x 256
// = 168 x 384, the 168 that the compiler gives a kernel of 384 threads (65536 / 384,
// a multiple of 8).
constexpr int kFewRegisters = 56, kManyRegisters = 224;

// Whether a block launched with this many registers to a thread has what its warpgroups
// take.  With fewer, the warpgroups that ask for more would wait for ever.
__host__ __device__ constexpr bool registers_suffice(int at_launch) {
    return at_launch * kPairThreads >= kFewRegisters * 128 + kManyRegisters * (kPairThreads - 128);
}

}  // namespace tr

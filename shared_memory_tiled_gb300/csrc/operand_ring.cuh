// How the warp that loads a ring of operand stages leaves it.  For the device and, so
// that the order can be walked without a GPU, the host.
#pragma once

#include <cstdint>

namespace tr {

// Block n of the contraction goes to stage n % STAGES.  Its loads complete phase
// n / STAGES of the stage's `full` barrier, the commit behind the matrix instructions
// that read it phase n / STAGES of its `empty` one.  A load or a commit that arrives
// after its block has left the SM would land in another block's shared memory, and
// the warp that loads waits for a commit only before it fills the stage again.  So,
// with `filled` blocks behind it, it waits for the last commit of each stage:
// released(stage, parity), false if that wait ran out.  Where one does not come (a warp
// that gave up), landed(stage, parity) waits for the loads instead.
template <int STAGES, typename Released, typename Landed>
__host__ __device__ __forceinline__ bool leave_ring(int64_t filled, const Released &released, const Landed &landed) {
    for (int64_t n = filled > STAGES ? filled - STAGES : 0; n < filled; ++n) {
        if (released(int(n % STAGES), uint32_t(n / STAGES) & 1u)) continue;
        for (; n < filled; ++n) landed(int(n % STAGES), uint32_t(n / STAGES) & 1u);
        return false;
    }
    return true;
}

}  // namespace tr

// Self-test of the bounded wait, in each unit whose kernels wait: one warp waits on an
// mbarrier phase that completes only if `arrive` is set (lane 0 arrives on it);
// otherwise the wait runs out after limit_ns and the unit's fault flag is raised
// exactly as in its kernels.  Nothing here can fault or hang: the wait is bounded.
#pragma once

#include "ptx.cuh"

namespace tr {

__device__ __forceinline__ void wait_selftest(unsigned *fault_flag, int arrive, uint64_t limit_ns) {
    __shared__ uint64_t bar;
    if (threadIdx.x == 0) {
        ptx::mbar_init(&bar, 1);
        ptx::fence_barrier_init();
    }
    __syncwarp();
    if (arrive && threadIdx.x == 0) ptx::mbar_arrive(&bar);
    const bool ok = ptx::mbar_wait_bounded(&bar, 0, limit_ns);
    if (__any_sync(0xffffffffu, !ok) && threadIdx.x == 0) atomicExch(fault_flag, 1u);
}

}  // namespace tr

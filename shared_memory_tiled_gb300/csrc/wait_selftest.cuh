// Self-test of the bounded wait, in each unit whose kernels wait: one warp waits on an
// mbarrier phase that completes only if `arrive` is set (lane 0 arrives on it);
// otherwise the wait runs out after limit_ns and the unit's fault flag is raised
// exactly as in its kernels.  Nothing here can fault or hang: the wait is bounded.
#pragma once

#include "ptx.cuh"
#include "tr_internal.h"

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
    if (__any_sync(0xffffffffu, !ok) && threadIdx.x == 0) atomicOr(fault_flag, kFaultWait);
}

// A unit's self-test and the host's reader of its fault flag g_fault_flag_<unit>.
#define TR_WAIT_UNIT(unit)                                                                              \
    __global__ void k_wait_selftest_##unit(int arrive, uint64_t limit_ns) {                             \
        wait_selftest(&g_fault_flag_##unit, arrive, limit_ns);                                          \
    }                                                                                                   \
    cudaError_t launch_wait_selftest_##unit(bool arrive, int64_t limit_ns, cudaStream_t stream) {       \
        k_wait_selftest_##unit<<<1, 32, 0, stream>>>(arrive ? 1 : 0, uint64_t(limit_ns));               \
        return cudaGetLastError();                                                                      \
    }                                                                                                   \
    cudaError_t read_and_clear_fault_##unit(unsigned *value) {                                          \
        const cudaError_t e = cudaMemcpyFromSymbol(value, g_fault_flag_##unit, sizeof(unsigned));       \
        if (e != cudaSuccess) return e;                                                                 \
        const unsigned zero = 0;                                                                        \
        return cudaMemcpyToSymbol(g_fault_flag_##unit, &zero, sizeof(unsigned));                        \
    }

}  // namespace tr

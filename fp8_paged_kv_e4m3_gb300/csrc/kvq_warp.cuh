// kvq_warp.cuh -- what a whole warp does together around the tcgen05 kernels'
// barriers and MMAs.
#pragma once

#include "kvq_device.cuh"

namespace kvq {

// one lane of a converged warp
__device__ __forceinline__ bool elect_one()
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}

// mbar_wait_bounded for a whole warp, all of whose lanes get the same answer.
// Every try is followed by a vote, so that the branch is the warp's: with each
// lane leaving mbar_wait_bounded's loop by itself, a wait for a phase long
// complete took 200 to 400 cycles in the tcgen05 kernel of the E2M1 cache.
__device__ __forceinline__ bool mbar_wait_warp(uint32_t bar, uint32_t parity, volatile int *abort, int32_t *err_flag)
{
    if (__builtin_expect(__all_sync(0xFFFFFFFFu, mbar_try_wait(bar, parity)), 1)) return true;
    uint64_t t0 = 0;
#pragma unroll 1
    for (uint32_t it = 1;; ++it) {
        if (__all_sync(0xFFFFFFFFu, mbar_try_wait(bar, parity))) return true;
        if ((it & 63u) == 0u) {
            if (__any_sync(0xFFFFFFFFu, *abort != 0)) return false;
            const uint64_t now = global_timer_ns();
            if (t0 == 0) t0 = now;
            if (__any_sync(0xFFFFFFFFu, now - t0 > kWaitLimitNs)) {
                *abort = 1;
                report(err_flag, KVQ_DEV_TIMEOUT);
                return false;
            }
        }
    }
}

}  // namespace kvq

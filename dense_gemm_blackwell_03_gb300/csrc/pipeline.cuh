// pipeline.cuh -- the bounded barrier wait of the operators' kernels.
#pragma once

#include "gemm_kernel.cuh"

namespace bwgemm {

// Bounded wait on an mbarrier phase: gives up after p.timeout_ns (recording
// `code` in the status word) or as soon as another role of this CTA gave up.
// The way through is a loop of a few instructions; the clock and the abort flag
// are looked at once in many probes, out of its way.
template <typename Params>
__device__ __forceinline__ bool pipe_wait(uint32_t bar, uint32_t parity, const Params& p, volatile uint32_t* abort_flag,
                                          uint32_t code)
{
    constexpr uint32_t kProbes = 2048;
    if (__builtin_expect(ptx::mbar_spin(bar, parity, kProbes), 1))
        return true;
    WaitClock clock;
#pragma unroll 1
    while (!ptx::mbar_spin(bar, parity, kProbes)) {
        if (*abort_flag)
            return false;
        if (clock.expired(p.timeout_ns)) {
            atomicOr(p.status, code);
            *abort_flag = 1u;
            return false;
        }
    }
    return true;
}

// The same for a converged warp, whose result is the same in every lane.  Nearly always the
// barrier's phase is complete or completes within the first probe; a vote and a uniform branch
// on that takes 109 cycles on a complete phase, pipe_wait with its vote 260 (its loop
// and its calls are kept apart lane by lane).
template <typename Params>
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, const Params& p, volatile uint32_t* abort_flag,
                                          uint32_t code)
{
    if (__all_sync(0xffffffffu, ptx::mbar_try_wait(bar, parity)))
        return true;
    return __all_sync(0xffffffffu, pipe_wait(bar, parity, p, abort_flag, code));
}

// Hand a TMEM accumulator that this warp has read (tcgen05.wait::ld done) back to
// the MMA warp of the pair's even CTA, or of this CTA.  What has to be ordered
// are the TMEM reads, which the tcgen05 fences on both sides order; the arrival
// itself is relaxed.
template <int CG>
__device__ __forceinline__ void hand_back(uint32_t bar, int lane)
{
    ptx::tc_fence_before_sync();
    __syncwarp();
    if (lane == 0) {
        if constexpr (CG == 1)
            ptx::mbar_arrive_relaxed(bar);
        else
            ptx::mbar_arrive_cluster_relaxed(ptx::map_to_cta(bar, 0));
    }
}

}  // namespace bwgemm

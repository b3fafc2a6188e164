// warp_wait.cuh -- what the kernels with warp roles share: arriving on and waiting
// for mbarriers as a whole warp within a time, and their rings. (Apart from
// ptx.cuh, which is among the sources of the sampling kernels: the committed
// counters of those are tied to their sources' hash.)
#pragma once

#include <cstdint>

#include "ptx.cuh"

namespace dst {

__device__ __forceinline__ void mbar_arrive(uint64_t* bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

__device__ __forceinline__ uint64_t now_ns()
{
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

// A whole warp waits for the phase of `bar` with the given parity until the
// global timer shows `until`. All of its lanes get the same answer, as what
// depends on it often is an instruction of the whole warp: each lane polls for
// itself, and as the time runs out some might see the phase and others not.
__device__ __forceinline__ bool mbar_wait_warp(uint64_t* bar, uint32_t parity, uint64_t until)
{
    for (uint32_t i = 0; i < (1u << 30); ++i) {
        if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
        if ((i & 63u) == 63u && __any_sync(0xffffffffu, now_ns() > until)) return false;
    }
    return false;
}

// True in one lane of a warp whose lanes are together.
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// A place in a ring of buffers and the parity of its phase.
struct RingPlace {
    uint32_t at, phase;
    __device__ __forceinline__ void next(uint32_t n)
    {
        if (++at == n) {
            at = 0;
            phase ^= 1u;
        }
    }
};

}  // namespace dst

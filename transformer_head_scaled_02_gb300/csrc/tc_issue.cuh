// tc_issue.cuh -- issuing tcgen05 work from a whole, converged warp.
//
// One thread issues an MMA, but where that thread runs alone (if (lane == 0) ...) the compiler has to move
// every descriptor from its registers to the uniform ones the instruction reads: about 100 cycles per
// MMA, more than a 128 x 64 product of 16 takes.  Here the warp stays together, waits and loop counters
// are the same in all lanes, and each instruction is predicated on the one elected lane.
#pragma once

#include "ptx.cuh"

namespace mha {

// 1 in one lane of the (converged) warp, always the same one.
__device__ __forceinline__ uint32_t elect_lane() {
    uint32_t e;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(e));
    return e;
}

// The same value in all lanes, as the compiler knows it: operands of MMAs computed from such values need no
// search for a common one.
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

// mbar_wait in less code (32 bits of the clock; giving up after another's abort records the status once more,
// which keeps the first): a kernel with thirty waits holds it thirty times between the instructions that run
// all the time, and the instruction cache is what its roles share.
__device__ __forceinline__ uint32_t globaltimer_lo() {
    uint32_t t;
    asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t));
    return t;
}

__device__ __forceinline__ bool lean_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* status) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint32_t t0 = globaltimer_lo();
    while (!mbar_try_wait_sleep(bar, parity, 100000u))
        if (*abort_flag || globaltimer_lo() - t0 > (uint32_t)kWaitLimitNs) {
            *abort_flag = 1;
            record_status(status, kStatusTimeout);
            return false;
        }
    return true;
}

// A wait with an outcome that is the same in all lanes.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* status) {
    return __all_sync(0xffffffffu, lean_wait(bar, parity, abort_flag, status));
}

__device__ __forceinline__ void mma_bf16_ss_elect(uint32_t elected, uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                                  uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(elected)
        : "memory");
}

__device__ __forceinline__ void mma_bf16_ts_elect(uint32_t elected, uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                                  uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(elected)
        : "memory");
}

__device__ __forceinline__ void tc_commit_elect(uint32_t elected, uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}\n" ::"r"(bar),
        "r"(elected)
        : "memory");
}

}  // namespace mha

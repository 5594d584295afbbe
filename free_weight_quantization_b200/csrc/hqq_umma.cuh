// hqq_umma.cuh -- mbarriers with bounded waits and the tcgen05 helpers that the tensor-core kernels
// share.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace {

constexpr uint32_t kMbarWaitLimit = 1u << 20;

// tcgen05 shared-memory matrix descriptor: start address, leading-dimension byte offset,
// stride byte offset, all in 16-byte units; descriptor version 1; layout type (0: no swizzle,
// 2: 128-byte swizzle)
__device__ __forceinline__ uint64_t umma_desc(uint32_t saddr, uint32_t lbo, uint32_t sbo, uint32_t layout) {
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)((lbo >> 4) & 0x3FFFu) << 16) |
           ((uint64_t)((sbo >> 4) & 0x3FFFu) << 32) | ((uint64_t)1 << 46) | ((uint64_t)layout << 61);
}

__device__ __forceinline__ void mbar_init(uint32_t addr, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(addr), "r"(count) : "memory");
}

// one test of the phase with the given parity
__device__ __forceinline__ bool mbar_try(uint32_t addr, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred P1;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 P1, [%1], %2;\n\t"
        "selp.b32 %0, 1, 0, P1;\n\t}"
        : "=r"(ok)
        : "r"(addr), "r"(parity)
        : "memory");
    return ok != 0;
}

// bounded wait for the phase with the given parity, out of line: the hot loops only pay for it
// when the first test fails; false if the phase did not complete in time
__device__ __noinline__ bool mbar_wait_slow(uint32_t addr, uint32_t parity) {
    for (uint32_t i = 0; i < kMbarWaitLimit; ++i) {
        if (mbar_try(addr, parity)) return true;
        if (i >= 4) __nanosleep(64);  // a waiting warp leaves the issue slots to the working ones
    }
    return false;
}

__device__ __forceinline__ bool mbar_wait(uint32_t addr, uint32_t parity) {
    return mbar_try(addr, parity) || mbar_wait_slow(addr, parity);
}

__device__ __forceinline__ void mbar_arrive(uint32_t addr) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(addr) : "memory");
}

__device__ __forceinline__ void umma_commit(uint32_t mbar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(mbar) : "memory");
}

}  // namespace

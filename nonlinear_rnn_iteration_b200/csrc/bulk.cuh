// bulk.cuh -- waits with a limit on mbarriers, and untiled bulk copies into
// shared memory.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "cluster.cuh"
#include "common.cuh"
#include "tma.cuh"

namespace pararnn {

constexpr uint64_t kWaitNs = 2000000000ull;

// a wait with a limit; after one that ran out of time the others are short
template <bool kPeers>
__device__ __forceinline__ void wait_bar(uint64_t* bar, uint32_t parity, bool& late) {
    if (kPeers ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity)) return;
    const uint64_t t0 = globaltimer_ns(), limit = late ? 1000000ull : kWaitNs;
    while (!(kPeers ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity)))
        if (globaltimer_ns() - t0 > limit) {
            late = true;
            return;
        }
}

// `bytes` from src to shared memory, counted on `bar`; all three multiples of 16
__device__ __forceinline__ void bulk_load(void* dst, uintptr_t src, unsigned bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

}  // namespace pararnn

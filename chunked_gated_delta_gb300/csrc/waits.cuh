// waits.cuh -- bounded waits on mbarriers, the election of one thread of a warp
// and the untiled bulk load (decode step, projection).
#pragma once
#include "common.cuh"
#include "ptx.cuh"

namespace kda {
namespace {

// Waits for the phase with this parity, for kWaitLimitNs at most (the clock is
// read after each thousand tries).  The phase before it must be over, and the
// one after it not: parity tells no more.
// CLUSTER: the arrivals may come from the other CTA of a pair.
template <bool CLUSTER = false>
__device__ __forceinline__ bool try_wait(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    if constexpr (CLUSTER)
        asm volatile(
            "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], "
            "%2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(ptx::smem_u32(bar)), "r"(parity)
            : "memory");
    else
        ok = ptx::mbar_try_wait(bar, parity);
    return ok != 0;
}
template <bool CLUSTER = false>
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, uint64_t limit_ns = kWaitLimitNs) {
    uint64_t t0 = 0;
    while (true) {
#pragma unroll 1
        for (int i = 0; i < 1024; ++i)
            if (try_wait<CLUSTER>(bar, parity)) return true;
        const uint64_t t = ptx::globaltimer_ns();
        if (t0 == 0) t0 = t;
        else if (t - t0 > limit_ns) return false;
    }
}
// One lane of a converged warp.  Unlike a test of the lane number it tells the
// compiler that a single thread runs what follows, so that TMA and tcgen05
// instructions take their operands from uniform registers without a loop.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// Bulk copy: 16-byte aligned, a multiple of 16 bytes.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
            ptx::smem_u32(dst)),
        "l"(src), "r"(bytes), "r"(ptx::smem_u32(bar))
        : "memory");
}

}  // namespace
}  // namespace kda

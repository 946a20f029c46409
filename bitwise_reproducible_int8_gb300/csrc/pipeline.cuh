// pipeline.cuh -- shared-memory barrier and tensor-copy helpers for the
// pipelined kernels (k_fwd_tc.cu, k_bwd_tma.cu).  Every wait is
// bounded: mbar_wait gives up after WAIT_CYCLES and returns false, and the
// caller records the failure in the device error word and unwinds.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace repro {

constexpr long long WAIT_CYCLES = 4000000000LL;   // ~2 s at the boost clock

__device__ __forceinline__ uint32_t su32(const void* p)
{
    return (uint32_t)__cvta_generic_to_shared(p);
}

__device__ __forceinline__ void mbar_init(uint64_t* b, uint32_t count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(su32(b)), "r"(count) : "memory");
}

__device__ __forceinline__ void mbar_expect_tx(uint64_t* b, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(su32(b)),
                 "r"(bytes)
                 : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint64_t* b)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(su32(b)) : "memory");
}

__device__ __forceinline__ bool mbar_test(uint64_t* b, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(su32(b)), "r"(parity)
        : "memory");
    return ok != 0;
}

// true once the phase with this parity has completed; false after the limit
__device__ __forceinline__ bool mbar_wait(uint64_t* b, uint32_t parity)
{
    const long long t0 = clock64();
    while (!mbar_test(b, parity)) {
        if (clock64() - t0 > WAIT_CYCLES)
            return false;
    }
    return true;
}

// The same by a whole warp: one outcome for all of its lanes, so that none leaves a loop whose other lanes
// go on to an instruction that takes the whole warp, and lane 0 can report for all
__device__ __forceinline__ bool mbar_wait_warp(uint64_t* b, uint32_t parity)
{
    if (__all_sync(0xffffffffu, mbar_test(b, parity)))   // mostly: no clock is read
        return true;
    return __all_sync(0xffffffffu, mbar_wait(b, parity));
}

__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* map, int x, int y,
                                            uint64_t* bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(su32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(su32(bar))
        : "memory");
}

// contiguous copy of `bytes` (a multiple of 16; both addresses 16-byte
// aligned) from global to shared memory, completing on `bar`
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar)
{
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
            su32(dst)),
        "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(su32(bar))
        : "memory");
}

} // namespace repro

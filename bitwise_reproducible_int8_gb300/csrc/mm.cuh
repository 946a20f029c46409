// mm.cuh -- what the paths of the product of codes share (k_matmul_i8.cu, k_matmul_few.cu): codes to
// fp16, and sums to outputs.
#pragma once

#include <cuda_fp16.h>

#include "elem.cuh"

namespace repro {

// four codes to two words of fp16 pairs, all exact, in 5 instructions (bf16's shorter significand takes
// 8): u = code + 128 below the bits of 1024, less 1152
__device__ __forceinline__ uint2 widen4(uint32_t c)
{
    const uint32_t u = c ^ 0x80808080u;
    const uint32_t lo = __byte_perm(u, 0x64646464u, 0x4140), hi = __byte_perm(u, 0x64646464u, 0x4342);   // u, 0x64, u, 0x64
    const __half2 off = __half2(__float2half_rn(-1152.0f), __float2half_rn(-1152.0f));
    const __half2 a = __hadd2(*reinterpret_cast<const __half2*>(&lo), off), b = __hadd2(*reinterpret_cast<const __half2*>(&hi), off);
    return make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

// what every path ends with
template <typename Y> __device__ __forceinline__ void put(Y* p, float v, bool accumulate)
{
    if (accumulate)
        v = fadd_ftz(to_f32<Y>(*p), v);
    *p = from_f32<Y>(v);
}

__device__ __forceinline__ float scaled(int acc, bool has_a, float sa, bool has_b, float sb)
{
    float v = __int2float_rn(acc);
    if (has_a)
        v = fmul_flush(v, sa);
    return has_b ? fmul_flush(v, sb) : v;
}

} // namespace repro

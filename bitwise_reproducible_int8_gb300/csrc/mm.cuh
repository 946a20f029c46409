// mm.cuh -- what the paths of the product of codes share (k_matmul_i8.cu, k_matmul_few.cu): codes to
// bf16, and sums to outputs.
#pragma once

#include <cuda_bf16.h>

#include "elem.cuh"

namespace repro {

// four codes to two words of bf16 pairs: 128 + low seven bits less 128 or 256, all exact
__device__ __forceinline__ uint2 widen4(uint32_t c)
{
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t b = __byte_perm(c, 0, i == 0 ? 0x4140 : 0x4342);      // code, 0, code, 0
        const uint32_t hi = (b & 0x007f007fu) | 0x43004300u, lo = (b & 0x00800080u) | 0x43004300u;
        const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&hi),
                                         *reinterpret_cast<const __nv_bfloat162*>(&lo));
        w[i] = *reinterpret_cast<const uint32_t*>(&d);
    }
    return make_uint2(w[0], w[1]);
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

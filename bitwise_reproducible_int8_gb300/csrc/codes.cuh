// codes.cuh -- 8-bit codes of values that share a scale: s = max |v| (/) 127 and
// code = clamp(round_half_even(v (/) s), -127, 127), the quotient correctly rounded.
//
// A division per value would take most of a kernel's instructions.  v (x) RN(1 / s) is within
// 2^-23 of the quotient relative to it (half a unit for the reciprocal, half for the product), so
// within 127 2^-23 < 2^-16 of it; unless it lies that near to a whole number and a half, both
// round to the same whole number.  A value that does is divided, and so is every value of a scale
// whose reciprocal is not a normal number away from the ends of the range.
#pragma once

#include "common.cuh"

namespace repro {

struct CodeScale {
    float s;        // the scale, flushed
    float inv;      // RN(1 / s), or NaN where values have to be divided
};

__device__ __forceinline__ CodeScale code_scale(float s)
{
    CodeScale c;
    c.s = flush(s);
    // reciprocals from 2^-100 to 2^100: neither they nor the products of |v| <= 127.5 s lose bits
    c.inv = s >= 0x1p-100f && s <= 0x1p100f ? __frcp_rn(s) : __int_as_float(0x7fc00000);
    return c;
}

// scale of the largest magnitude m (whose bits order as m does)
__device__ __forceinline__ CodeScale code_scale_of_max(float m) { return code_scale(flush(__fdiv_rn(m, 127.0f))); }

static __device__ __noinline__ int code_by_division(float v, float s)
{
    if (s == 0.0f)
        return 0;
    const int q = __float2int_rn(__fdiv_rn(v, s));   // NaN to 0, saturating
    return q > 127 ? 127 : q < -127 ? -127 : q;
}

// codes of four values (flushed), packed; by one scale or by one each
__device__ __forceinline__ uint32_t codes4_by(const float (&v)[4], const CodeScale (&c)[4])
{
    constexpr float M = 12582912.0f;   // 1.5 2^23: adding it rounds to a whole number, ties to even
    uint32_t q[4];
    bool near = false;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float y = __fmul_rn(v[e], c[e].inv), r = __fadd_rn(y, M);
        q[e] = __float_as_uint(r);
        // within 2^-15 of a whole number and a half, or a NaN
        near |= !(fabsf(__fsub_rn(y, __fsub_rn(r, M))) < 0.5f - 0x1p-15f);
    }
    if (near) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            q[e] = (uint32_t)code_by_division(v[e], c[e].s);
    }
    return __byte_perm(__byte_perm(q[0], q[1], 0x0040), __byte_perm(q[2], q[3], 0x0040), 0x5410);
}

__device__ __forceinline__ uint32_t codes4(const float (&v)[4], const CodeScale& c)
{
    const CodeScale all[4] = {c, c, c, c};
    return codes4_by(v, all);
}

} // namespace repro

// codes.cuh -- 8-bit codes of values that share a scale: s = max |v| (/) 127 and
// code = clamp(round_half_even(v (/) s), -127, 127), the quotient correctly rounded.
//
// A division per value would take most of a kernel's instructions.  With r the hardware's reciprocal
// of s (within 2^-23 of 1 / s, relative), v (x) r is within 1.5 2^-23 of the quotient, so within 127.5
// 1.5 2^-23 < 2^-15 of it absolutely; unless it lies that near to a whole number and a half, both round
// to the same whole number.  A value that does is divided, and so is every value of a scale outside
// 2^-100 .. 2^100.
#pragma once

#include "common.cuh"

namespace repro {

struct CodeScale {
    float s;        // the scale, flushed
    float inv;      // about 1 / s, or NaN where values have to be divided
};

// The scale m (/) 127 of the largest magnitude m.  RN(z m + RN(z' m)) with z = RN(1 / 127), z' =
// RN(1 / 127 - z) is the correctly rounded quotient of every m whose products are normal (Brisebarre,
// Muller and Raina, "Accelerating correctly rounded floating-point division when the divisor is known
// in advance"; every mantissa checked: tests/div127_check.c).
__device__ __forceinline__ CodeScale code_scale_of_max(float m)
{
    CodeScale c;
    if (m >= 0x1p-90f && m <= 0x1p100f) {
        c.s = __fmaf_rn(0x1.020408p-7f, m, __fmul_rn(0x1.020408p-35f, m));
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(c.inv) : "f"(c.s));
    } else {
        c.s = flush(__fdiv_rn(flush(m), 127.0f));
        c.inv = __int_as_float(0x7fc00000);
    }
    return c;
}

__device__ __forceinline__ int code_by_division(float v, float s)
{
    if (s == 0.0f)
        return 0;
    const int q = __float2int_rn(__fdiv_rn(flush(v), s));   // NaN to 0, saturating
    return q > 127 ? 127 : q < -127 ? -127 : q;
}

// codes of four values, packed, by a scale each; far: none of them has to be divided.  A subnormal
// value is read as zero: by the division, and beside a scale of 2^-97 or more by itself
__device__ __forceinline__ uint32_t codes4_near(const float (&v)[4], const CodeScale (&c)[4], bool& far)
{
    constexpr float M = 12582912.0f;   // 1.5 2^23: adding it rounds to a whole number, ties to even
    uint32_t q[4];
    far = true;
#pragma unroll
    for (int e = 0; e < 4; e += 2) {
        const unsigned long long y = fmul2_rn(pack2(v[e], v[e + 1]), pack2(c[e].inv, c[e + 1].inv));
        const unsigned long long r = fadd2_ftz(y, pack2(M, M));
        const unsigned long long d = ffma2_rn(fadd2_ftz(r, pack2(-M, -M)), pack2(-1.0f, -1.0f), y);   // y - its whole number, exact
        float r0, r1, d0, d1;
        unpack2(r, r0, r1);
        unpack2(d, d0, d1);
        q[e] = __float_as_uint(r0);
        q[e + 1] = __float_as_uint(r1);
        far = far && fabsf(d0) < 0.5f - 0x1p-15f && fabsf(d1) < 0.5f - 0x1p-15f;   // not of a NaN
    }
    return __byte_perm(__byte_perm(q[0], q[1], 0x0040), __byte_perm(q[2], q[3], 0x0040), 0x5410);
}

__device__ __forceinline__ uint32_t codes4_divided(const float (&v)[4], const CodeScale (&c)[4])
{
    uint32_t q = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e)
        q |= (uint32_t)(code_by_division(v[e], c[e].s) & 0xff) << (8 * e);
    return q;
}

// by one scale
__device__ __forceinline__ uint32_t codes4(const float (&v)[4], const CodeScale& c)
{
    const CodeScale all[4] = {c, c, c, c};
    bool far;
    const uint32_t q = codes4_near(v, all, far);
    return far ? q : codes4_divided(v, all);
}

} // namespace repro

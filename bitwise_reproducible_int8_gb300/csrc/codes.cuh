// codes.cuh -- 8-bit codes of values that share a scale: s = max |v| (/) 127 and
// code = clamp(round_half_even(v (/) s), -127, 127), the quotient correctly rounded.
//
// A division per value would take most of a kernel's instructions.  With r = RN(1 / s) (the hardware's
// reciprocal and one Newton step; P. Markstein, "Computation of elementary functions on the IBM RISC
// System/6000 processor", 1990), y = RN(v (x) r) and q = RN(y + r RN(v - y s)), q is within 2^-46 of the
// quotient before its last rounding, and rounds to the same whole number as the rounded quotient: where
// the two could part there are a few thousand scales' significands, and for none of them do they
// (tests/codes_check.c, which also derives the bound).  Values of a scale outside 2^-67 .. 2^94 are
// divided.
#pragma once

#include "common.cuh"

namespace repro {

struct CodeScale {
    float s;        // the scale, flushed
    float inv;      // RN(1 / s), or NaN where values have to be divided
};

// The scale m (/) 127 of the largest magnitude m.  RN(z m + RN(z' m)) with z = RN(1 / 127), z' =
// RN(1 / 127 - z) is the correctly rounded quotient of every m whose products are normal (Brisebarre,
// Muller and Raina, "Accelerating correctly rounded floating-point division when the divisor is known
// in advance"; every mantissa checked: tests/div127_check.c).
__device__ __forceinline__ CodeScale code_scale_of_max(float m)
{
    CodeScale c;
    if (m >= 0x1p-60f && m <= 0x1p100f) {
        float r;
        c.s = __fmaf_rn(0x1.020408p-7f, m, __fmul_rn(0x1.020408p-35f, m));
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(c.s));
        c.inv = __fmaf_rn(r, __fmaf_rn(-c.s, r, 1.0f), r);
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

// codes of four values, packed, by a scale each; false where a value is a NaN, or one's scale has no
// reciprocal: those have to be divided.  A subnormal value is read as zero: by the division, and beside a
// scale of 2^-67 or more by itself
__device__ __forceinline__ bool codes4(const float (&v)[4], const CodeScale (&c)[4], uint32_t& codes)
{
    constexpr float M = 12582912.0f;   // 1.5 2^23: adding it rounds to a whole number, ties to even
    uint32_t q[4];
#pragma unroll
    for (int e = 0; e < 4; e += 2) {
        const unsigned long long x = pack2(v[e], v[e + 1]), r = pack2(c[e].inv, c[e + 1].inv), y = fmul2_rn(x, r);
        const unsigned long long t = ffma2_rn(ffma2_rn(y, pack2(-c[e].s, -c[e + 1].s), x), r, y);
        float r0, r1;
        unpack2(fadd2_ftz(t, pack2(M, M)), r0, r1);
        q[e] = __float_as_uint(r0);
        q[e + 1] = __float_as_uint(r1);
    }
    codes = __byte_perm(__byte_perm(q[0], q[1], 0x0040), __byte_perm(q[2], q[3], 0x0040), 0x5410);
    return (q[0] | q[1] | q[2] | q[3]) < 0x7f800000u;   // no NaN: the others lie between 2^23 and 2^24
}

__device__ __forceinline__ uint32_t codes4_divided(const float (&v)[4], const CodeScale (&c)[4])
{
    uint32_t q = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e)
        q |= (uint32_t)(code_by_division(v[e], c[e].s) & 0xff) << (8 * e);
    return q;
}

} // namespace repro

// expr.cuh -- exp_r, the e^x of the attention's softmax and of the gated activation, fixed in
// every operation: Cody-Waite range reduction (ln 2 = 355/512 + RN(ln 2 - 355/512)), degree-7
// Taylor polynomial in Horner form with RN(1/n!) coefficients, exact scaling by 2^k.
#pragma once

#include "common.cuh"

namespace repro {

// e^x of one value
__device__ __forceinline__ float exp_r(float x)
{
    x = flush(x);
    const float kf = rintf(fmul_flush(x, 0x1.715476p+0f));
    const float r = fadd_ftz(fadd_ftz(x, -fmul_flush(kf, 0x1.63p-1f)),
                             -fmul_flush(kf, -0x1.bd0106p-13f));
    float p = 0x1.a01a02p-13f;
    p = fadd_ftz(fmul_rn(p, r), 0x1.6c16c2p-10f);
    p = fadd_ftz(fmul_rn(p, r), 0x1.111112p-7f);
    p = fadd_ftz(fmul_rn(p, r), 0x1.555556p-5f);
    p = fadd_ftz(fmul_rn(p, r), 0x1.555556p-3f);
    p = fadd_ftz(fmul_rn(p, r), 0.5f);
    p = fadd_ftz(fmul_rn(p, r), 1.0f);
    p = fadd_ftz(fmul_rn(p, r), 1.0f);
    if (kf < -126.0f)
        return 0.0f;
    if (kf > 254.0f)
        return __int_as_float(0x7f800000);
    const int k = (int)kf;
    if (k > 127)
        return flush(fmul_rn(fmul_rn(p, 0x1p127f), __int_as_float((k - 127 + 127) << 23)));
    return flush(fmul_rn(p, __int_as_float((k + 127) << 23)));
}

// e^x of two lanes: the same operations as exp_r, lane by lane, with the
// reduction and the polynomial on packed pairs
__device__ __forceinline__ float exp_scale(float p, float kf)
{
    if (kf < -126.0f)
        return 0.0f;
    if (kf > 254.0f)
        return __int_as_float(0x7f800000);
    const int k = (int)kf;
    if (k > 127)
        return flush(fmul_rn(fmul_rn(p, 0x1p127f), __int_as_float((k - 127 + 127) << 23)));
    return flush(fmul_rn(p, __int_as_float((k + 127) << 23)));
}

__device__ __forceinline__ unsigned long long exp_r2(unsigned long long x)
{
    const unsigned long long z = pack2(-0.0f, -0.0f);
    x = fadd2_ftz(x, z);
    float t0, t1;
    unpack2(fadd2_ftz(fmul2_rn(x, pack2(0x1.715476p+0f, 0x1.715476p+0f)), z), t0, t1);
    const float k0 = rintf(t0), k1 = rintf(t1);
    const unsigned long long kf = pack2(k0, k1);
    // x (-) RN(kf c1), then (-) RN(kf c2); the negated products are RN(kf (-c))
    const unsigned long long r = fadd2_ftz(fadd2_ftz(x, fadd2_ftz(fmul2_rn(kf, pack2(-0x1.63p-1f, -0x1.63p-1f)), z)),
                            fadd2_ftz(fmul2_rn(kf, pack2(0x1.bd0106p-13f, 0x1.bd0106p-13f)), z));
    unsigned long long p = pack2(0x1.a01a02p-13f, 0x1.a01a02p-13f);
    p = fadd2_ftz(fmul2_rn(p, r), pack2(0x1.6c16c2p-10f, 0x1.6c16c2p-10f));
    p = fadd2_ftz(fmul2_rn(p, r), pack2(0x1.111112p-7f, 0x1.111112p-7f));
    p = fadd2_ftz(fmul2_rn(p, r), pack2(0x1.555556p-5f, 0x1.555556p-5f));
    p = fadd2_ftz(fmul2_rn(p, r), pack2(0x1.555556p-3f, 0x1.555556p-3f));
    p = fadd2_ftz(fmul2_rn(p, r), pack2(0.5f, 0.5f));
    p = fadd2_ftz(fmul2_rn(p, r), pack2(1.0f, 1.0f));
    p = fadd2_ftz(fmul2_rn(p, r), pack2(1.0f, 1.0f));
    // 2^k exactly as a normal float for -126 <= k <= 127: both lanes scale in
    // one packed multiply; any other lane takes exp_scale's branches
    if (k0 >= -126.0f && k0 <= 127.0f && k1 >= -126.0f && k1 <= 127.0f) {
        const unsigned long long sc = pack2(__int_as_float(((int)k0 + 127) << 23), __int_as_float(((int)k1 + 127) << 23));
        return fadd2_ftz(fmul2_rn(p, sc), z);
    }
    float p0, p1;
    unpack2(p, p0, p1);
    return pack2(exp_scale(p0, k0), exp_scale(p1, k1));
}

// exp_r of two lanes whose arguments are not above 0 (a NaN counts as far below: 0), in fewer
// operations and with the same bits: 2^k is an addition to the exponent, k the low bits of
// x log2 e + 1.5 2^23; below e^-100 nothing is left, so the argument may stop there; and the
// flushes that can change nothing are left out (k and its products are 0 or normal)
__device__ __forceinline__ unsigned long long exp_r2_neg(float x0, float x1)
{
    const unsigned long long M = pack2(12582912.0f, 12582912.0f);
    const unsigned long long x = pack2(fmaxf(x0, -100.0f), fmaxf(x1, -100.0f));
    const unsigned long long t = fadd2_ftz(fmul2_rn(x, pack2(0x1.715476p+0f, 0x1.715476p+0f)), M);
    const unsigned long long kf = fadd2_ftz(t, pack2(-12582912.0f, -12582912.0f));
    const unsigned long long r = fadd2_ftz(fadd2_ftz(x, fmul2_rn(kf, pack2(-0x1.63p-1f, -0x1.63p-1f))),
                                           fmul2_rn(kf, pack2(0x1.bd0106p-13f, 0x1.bd0106p-13f)));
    unsigned long long p = pack2(0x1.a01a02p-13f, 0x1.a01a02p-13f);
    p = fadd2_ftz(fmul2_rn(p, r), pack2(0x1.6c16c2p-10f, 0x1.6c16c2p-10f));
    p = fadd2_ftz(fmul2_rn(p, r), pack2(0x1.111112p-7f, 0x1.111112p-7f));
    p = fadd2_ftz(fmul2_rn(p, r), pack2(0x1.555556p-5f, 0x1.555556p-5f));
    p = fadd2_ftz(fmul2_rn(p, r), pack2(0x1.555556p-3f, 0x1.555556p-3f));
    p = fadd2_ftz(fmul2_rn(p, r), pack2(0.5f, 0.5f));
    p = fadd2_ftz(fmul2_rn(p, r), pack2(1.0f, 1.0f));
    p = fadd2_ftz(fmul2_rn(p, r), pack2(1.0f, 1.0f));
    float p0, p1, t0, t1, k0, k1;
    unpack2(p, p0, p1);
    unpack2(t, t0, t1);
    unpack2(kf, k0, k1);
    // k = -126 with a factor below 1 is subnormal, and below -126 all is
    p0 = k0 >= -126.0f ? __int_as_float(__float_as_int(p0) + (__float_as_int(t0) << 23)) : 0.0f;
    p1 = k1 >= -126.0f ? __int_as_float(__float_as_int(p1) + (__float_as_int(t1) << 23)) : 0.0f;
    return fadd2_ftz(pack2(p0, p1), pack2(-0.0f, -0.0f));
}

} // namespace repro

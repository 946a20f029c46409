/* The 8-bit codes' quotient without a division: y = RN(v r), q = RN(y + r RN(v - y s)), r = RN(1 / s).
 * q is RN((v / s) (1 + t)), |t| < 2^-46, and its rounding to a whole number can differ from that of
 * RN(v / s) only where v / s lies that near to B = k + 1/2 +- half a last place of k + 1/2.  With
 * s = S 2^i and E = floor(log2(k + 1/2)) the distance v - B s is a multiple n of 2^(i+E-24), where v is
 * one of 2^(i+E): n = -S ((2k + 1) 2^(23-E) +- 1) modulo 2^24, the factor odd, so each n has one S, and
 * |n| <= 8 is what the bound leaves.  Here: every k, both signs, |n| <= 64, against the division; and,
 * for scales of every kind, values about each half, and others. */
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

static float of(uint32_t b)
{
    float x;
    memcpy(&x, &b, 4);
    return x;
}

static uint32_t bits(float x)
{
    uint32_t b;
    memcpy(&b, &x, 4);
    return b;
}

static int by_division(float v, float s) { return (int)rintf(v / s); }

static int by_product(float v, float s, float r)
{
    const float y = v * r, d = fmaf(y, -s, v), q = fmaf(d, r, y);
    return (int8_t)(bits(q + 12582912.0f) & 0xff);
}

static uint64_t state = 88172645463325252ull;
static uint32_t next(void)
{
    state ^= state << 13;
    state ^= state >> 7;
    state ^= state << 17;
    return (uint32_t)(state >> 20);
}

static int check(float v, float s)
{
    const float r = 1.0f / s;
    if (fabsf(v) > 127.0f * s)
        return 0;
    if (by_product(v, s, r) != by_division(v, s) || by_product(-v, s, r) != -by_division(v, s)) {
        printf("v %a s %a: %d, not %d\n", v, s, by_product(v, s, r), by_division(v, s));
        return 1;
    }
    return 0;
}

int main(void)
{
    const int exponents[] = {127 - 67, 120, 127, 127 + 93};
    long near = 0;
    for (int k = 0; k < 127; ++k) {
        int E = 0;
        while (k >= 1 && (2 << E) <= k)
            ++E;
        if (k == 0)
            E = -1;
        for (int sign = -1; sign <= 1; sign += 2) {
            const uint32_t f = (uint32_t)((2 * k + 1) << (23 - E)) + (uint32_t)sign;   /* odd */
            uint32_t inverse = f;
            for (int i = 0; i < 5; ++i)
                inverse *= 2 - f * inverse;
            if (f * inverse != 1)
                return 2;
            for (int n = -64; n <= 64; ++n) {
                const uint32_t S = (uint32_t)-n * inverse & 0xffffffu;
                if (S < 0x800000u)
                    continue;
                ++near;
                for (int x = 0; x < 4; ++x) {
                    const float s = of((uint32_t)exponents[x] << 23 | (S & 0x7fffffu));
                    const double B = k + 0.5 + sign * ldexp(1.0, E - 24);
                    const float at = (float)(B * s);
                    for (int e = -3; e <= 3; ++e)
                        if (check(of(bits(at) + e), s))
                            return 1;
                }
            }
        }
    }
    if (near < 10000)
        return 2;
    for (int n = 0; n < 6000; ++n) {
        /* significands of few bits (a bf16 maximum by 127, whole numbers), all ones, and any */
        const uint32_t m = n < 128 ? (uint32_t)n << 16 : n < 140 ? 0x7fffffu - (n - 128) : n < 152 ? (uint32_t)(n - 140) : next() & 0x7fffffu;
        const float s0 = of((uint32_t)exponents[n & 3] << 23 | m);
        for (int kind = 0; kind < 2; ++kind) {
            const float s = kind || s0 / 127.0f < 0x1p-67f ? s0 : s0 / 127.0f;
            for (int k = 0; k < 127; ++k) {
                const float at = (float)((k + 0.5) * (double)s);
                for (int e = -12; e <= 12; ++e)
                    if (check(of(bits(at) + e), s))
                        return 1;
            }
            for (int i = 0; i < 100; ++i)
                if (check((float)(next() % 127000001u) * 1e-6f * s, s) || check(of(bits(127.0f * s) - i), s) || check(i * s, s) ||
                    check(of((uint32_t)i), s))
                    return 1;
        }
    }
    return 0;
}

/* Every significand: RN(z x + RN(z' x)), z = RN(1/127), z' = RN(1/127 - z), against x / 127, at an
 * exponent and at the two ends of the range that the 8-bit codes use it in. */
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

int main(void)
{
    const float zh = (float)(1.0 / 127.0), zl = (float)(1.0 / 127.0 - (double)zh);
    const int exponents[] = {127 - 90, 127, 127 + 99};
    if (zh != 0x1.020408p-7f || zl != 0x1.020408p-35f)
        return 1;
    for (int k = 0; k < 3; ++k)
        for (uint32_t m = 0; m < (1u << 23); ++m) {
            const uint32_t b = ((uint32_t)exponents[k] << 23) | m;
            float x;
            memcpy(&x, &b, 4);
            if (fmaf(zh, x, zl * x) != x / 127.0f) {
                printf("%a\n", x);
                return 1;
            }
        }
    return 0;
}

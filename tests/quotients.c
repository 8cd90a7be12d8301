/* The quotients that 8-bit codes are rounded from, and the scales (rows_out.h's
 * `quotients` and `scale_of`), against the divided ones: one IEEE operation per
 * written operation. Significands say it all: neither side leaves the normal range. */
#include <math.h>
#include <stdint.h>

static int side(float q, float mid) { return (q > mid) - (q < mid); }

/* For s = significand / 2^23 in [first, last), each midpoint m / 2^j in [1, 2) with m
 * odd and below 2^bits, and the nine x nearest to its product with s: how many
 * quotients lie on another side of the midpoint than x / s does. steps: remainders
 * taken (0: x times the reciprocal). */
long long other_sides(long first, long last, int bits, int steps)
{
    long long off = 0;
#pragma omp parallel for reduction(+ : off) schedule(static)
    for (long n = first; n < last; ++n) {
        const float s = (float)n * 0x1p-23f, r = 1.0f / s;
        for (int m = 1; m < 1 << bits; m += 2) {
            int j = 0;
            while (m >> (j + 1))
                ++j;
            const float mid = (float)m / (float)(1 << j);
            const float at = (float)((double)mid * (double)s);   /* exact before this rounding */
            uint32_t b;
            __builtin_memcpy(&b, &at, 4);
            int bad = 0;
            for (int d = -4; d <= 4; ++d) {
                const uint32_t xb = b + (uint32_t)d;
                float x;
                __builtin_memcpy(&x, &xb, 4);
                float q = x * r;
                for (int k = 0; k < steps; ++k)
                    q = fmaf(fmaf(-q, s, x), r, q);
                bad += side(q, mid) != side(x / s, mid);
            }
            off += bad;
        }
    }
    return off;
}

/* All significands of a block's maximum: how many max / c differ from the divided one. */
long long other_scales(float c, int steps)
{
    long long off = 0;
    const float r = 1.0f / c;
#pragma omp parallel for reduction(+ : off) schedule(static)
    for (long n = 1 << 23; n < 1 << 24; ++n) {
        const float max = (float)n * 0x1p-23f;
        float q = max * r;
        for (int k = 0; k < steps; ++k)
            q = fmaf(fmaf(-q, c, max), r, q);
        off += q != max / c;
    }
    return off;
}

// Host build of the quotient by which fp32 values become codes (w4a8_int8_gemm_amd/csrc/f8_rule.h and
// quant_rule.h), against the division where it is hardest.  Test code only.
#include <math.h>
#include <stdint.h>

#include "../../w4a8_int8_gemm_amd/csrc/f8_rule.h"

namespace {

// a^-1 modulo 2^64 for odd a
uint64_t inverse(uint64_t a)
{
    uint64_t x = a;
    for (int i = 0; i < 6; ++i)
        x *= 2 - a * x;
    return x;
}

long differ(float x, float s, float r)
{
    const float q = x / s;
    return (w4a8::f8_quotient(x, s, r) != q) + (w4a8::quant_div_corrected(x, s, r) != q);
}

// as the kernels: the reciprocal says whether both sides are lifted
float quotient(float x, float s)
{
    const float r = w4a8::f8_reciprocal(s);
    return r < 0.0f ? w4a8::f8_quotient(x * w4a8::kF8Lift, s * w4a8::kF8Lift, -r) : w4a8::f8_quotient(x, s, r);
}

}  // namespace

extern "C" {

// With 24-bit integers X and S for x and s, 2^k X / S lies between 2^23 and 2^24 for k = 23 (X >= S) or
// 24, and D = X 2^(k + 1) - (2 Q + 1) S is how far it is from the middle of Q and Q + 1, in units of
// 1 / (2 S).  All pairs with 0 < |D| <= 8, S in [lo, hi); and all with |X - S| <= 8.  How many quotients
// differ from the division.
long shim_hard(long lo, long hi, long *tried)
{
    long bad = 0;
    for (uint64_t S = (uint64_t)lo; S < (uint64_t)hi; ++S) {
        const float s = (float)S, r = 1.0f / s;
        for (int d = -8; d <= 8; ++d) {
            const int64_t X = (int64_t)S + d;
            if (X >= (1 << 23) && X < (1 << 24))
                bad += differ((float)X, s, r), ++*tried;
        }
        const int twos = __builtin_ctzll(S);               // D is a multiple of them, by an odd number
        if (twos > 3)
            continue;
        const uint64_t inv = inverse(S >> twos);
        for (int k = 23; k <= 24; ++k)
            for (int d = -8; d <= 8; ++d) {
                if (d == 0 || d % (1 << twos) != 0 || (d / (1 << twos)) % 2 == 0)
                    continue;
                const uint64_t mod = uint64_t(1) << (k + 1 - twos);
                for (uint64_t odd = ((uint64_t)(int64_t)(-d / (1 << twos)) * inv) & (mod - 1); odd < (1u << 25); odd += mod) {
                    if (odd < (1u << 24))
                        continue;
                    const uint64_t X = (odd * S + (uint64_t)(int64_t)d) >> (k + 1);
                    if (X < (1u << 23) || X >= (1u << 24) || (k == 23) != (X >= S))
                        continue;
                    bad += differ((float)X, s, r), ++*tried;
                }
            }
    }
    return bad;
}

// Quotients of n pairs: as the kernels take them, and with s as it is.
void shim_quotients(const float *x, const float *s, float *lifted, float *plain, float *division, long n)
{
    for (long i = 0; i < n; ++i) {
        lifted[i] = quotient(x[i], s[i]);
        plain[i] = w4a8::f8_quotient(x[i], s[i], 1.0f / s[i]);
        division[i] = x[i] / s[i];
    }
}

float shim_reciprocal(float s) { return w4a8::f8_reciprocal(s); }

}

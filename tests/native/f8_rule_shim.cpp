// Host build of the e4m3 rule (w4a8_int8_gemm_amd/csrc/f8_rule.h), so that the CPU test suite can
// check the kernels' quotient against the division on every fp16 input.  Test code only.
#include <math.h>
#include <stdint.h>

#include "../../w4a8_int8_gemm_amd/csrc/f8_rule.h"

static float h2f_bits(uint16_t h)
{
    const int e = (h >> 10) & 0x1f, m = h & 0x3ff;
    return e == 0 ? ldexpf((float)m, -24) : ldexpf((float)(m | 0x400), e - 25);
}

extern "C" {

// Every fp16 amax with bits in [lo, hi) and every fp16 x in [0, amax]: how many quotients differ from
// x / s (the rule is odd in x), and how many do without the correction step.
long shim_quotients(int lo, int hi, long *uncorrected)
{
    long bad = 0;
    for (int ab = lo; ab < hi; ++ab) {
        const float s = w4a8::f8_scale(h2f_bits((uint16_t)ab));
        const float r = 1.0f / s;
        for (int xb = 0; xb <= ab; ++xb) {
            const float x = h2f_bits((uint16_t)xb);
            bad += w4a8::f8_quotient(x, s, r) != x / s;
            *uncorrected += x * r != x / s;
        }
    }
    return bad;
}

float shim_quotient(float x, float s) { return w4a8::f8_quotient(x, s, 1.0f / s); }

float shim_scale(float amax) { return w4a8::f8_scale(amax); }

}

// Host build of the gated product's activation (w4a8_int8_gemm_amd/csrc/f8_rule.h), with an exponential and a
// reciprocal that are rounded to fp32 and then moved by whole units in the last place.  Test code only.
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "../../w4a8_int8_gemm_amd/csrc/f8_rule.h"

static float moved(float v, int units)
{
    for (; units > 0 && v < INFINITY; --units)
        v = nextafterf(v, INFINITY);
    for (; units < 0 && v > 0.0f; ++units)
        v = nextafterf(v, 0.0f);
    return v;
}

extern "C" void shim_activation(const float *g, float *out, long n, int gelu, int exp_units, int rcp_units)
{
    for (long i = 0; i < n; ++i)
        out[i] = w4a8::f8_activation_steps(
            g[i], gelu, [=](float x) { return moved((float)exp2((double)x), exp_units); },
            [=](float x) { return moved(1.0f / x, rcp_units); });
}

// Device helpers of the 8-bit floating point kernels (gfx950).
#pragma once

#include "device_common.hpp"
#include "f8_rule.h"

namespace w4a8 {

typedef int v8i __attribute__((ext_vector_type(8)));

// A block's scale and its reciprocal from the largest |v|, as bits.
__device__ __forceinline__ void f8_block_scale(uint32_t amax_bits, float &s, float &r)
{
    s = amax_bits >= 0x7f800000u ? __uint_as_float(0x7fc00000u) : f8_scale(__uint_as_float(amax_bits));
    r = s > 0.0f ? 1.0f / s : 0.0f;      // zero codes for s = 0 and s = NaN
}

// Four values' codes in one dword, the first lowest.  With r = 0 the codes
// are 0 whatever the values are.
__device__ __forceinline__ uint32_t f8_codes4(float a, float b, float c, float d, float s, float r)
{
    if (r == 0.0f)
        return 0u;
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(f8_quotient(a, s, r), f8_quotient(b, s, r), 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(f8_quotient(c, s, r), f8_quotient(d, s, r), w, true);
    return (uint32_t)w;
}

// silu(g) = g / (1 + e^-g); gelu in its tanh form, 0.5 g (1 + tanh z) =
// g / (1 + e^-2z) with z = sqrt(2 / pi) (g + 0.044715 g^3).  The exponential
// and the reciprocal are the hardware's (one step of fp32 each, and the
// rounded argument: about 2^-22 of the result relative for |g| up to 30, far
// below the output's own rounding); e^-g overflows to infinity for very
// negative g, which gives -0.
__device__ __forceinline__ float f8_activation(float g, int gelu)
{
    float t = g;
    if (gelu)
        t = 1.5957691216057308f * fmaf(0.044715f * g, g * g, g);
    const float e = __builtin_amdgcn_exp2f(-1.4426950408889634f * t);
    return g * __builtin_amdgcn_rcpf(1.0f + e);
}

}  // namespace w4a8

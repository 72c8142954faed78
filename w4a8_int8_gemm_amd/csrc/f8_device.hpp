// Device helpers of the 8-bit floating point kernels (gfx950).
//
// The products use __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4 with its own
// scales at 1: 128 of K in one instruction, which is one block, so that each
// result meets its two scales once and is added in fp32.  Inside, the unit
// aligns eight consecutive products to the largest and drops what lies below
// 2^-13 of its power of two (measured).  Seven may lose that much: up to 7 2^-13
// of the largest of eight, 8.5e-4 of the sum of magnitudes if every eight are
// so (fp16's own half step is 4.9e-4), and of a sum that cancels any part.  It
// takes seven products of a size 2^-13 of their neighbour's; as seen against
// exact sums (rms of the result; largest share of the sum of magnitudes): rows
// quantised from Gaussian values 1.4e-5 and 1.8e-5, with one channel 20 times
// the others 1.8e-5 and 8e-5, 200 times 4.3e-5 and 2.2e-4, codes of every size
// 5.1e-5 and 2.1e-4.  The 16 x 16 x 32 instruction for e4m3 aligns alike and has
// half the rate (2445 against 4770 TFLOP/s); codes widened to fp16 in its fp16
// form are exact to fp32, at that rate and with their widening besides.
#pragma once

#include "device_common.hpp"
#include "f8_rule.h"

namespace w4a8 {

typedef int v8i __attribute__((ext_vector_type(8)));

// A block's scale and its reciprocal (f8_reciprocal) from the largest |v|, as
// bits.  SMALL: s may lie below 2^-90 (of fp16 values it is 0 or above 2^-33).
template <bool SMALL = true>
__device__ __forceinline__ void f8_block_scale(uint32_t amax_bits, float &s, float &r)
{
    s = amax_bits >= 0x7f800000u ? __uint_as_float(0x7fc00000u) : f8_scale(__uint_as_float(amax_bits));
    r = SMALL ? f8_reciprocal(s) : s > 0.0f ? 1.0f / s : 0.0f;
}

// Four values' codes in one dword, the first lowest.  With r = 0 the codes
// are 0 whatever the values are.
template <bool SMALL = true>
__device__ __forceinline__ uint32_t f8_codes4(float a, float b, float c, float d, float s, float r)
{
    if (r == 0.0f)
        return 0u;
    if (SMALL && __builtin_expect(r < 0.0f, 0)) {
        a *= kF8Lift, b *= kF8Lift, c *= kF8Lift, d *= kF8Lift, s *= kF8Lift, r = -r;
    }
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(f8_quotient(a, s, r), f8_quotient(b, s, r), 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(f8_quotient(c, s, r), f8_quotient(d, s, r), w, true);
    return (uint32_t)w;
}

// The gated product's activation by the hardware's exponential and reciprocal
// (f8_rule.h has the steps and how far off they are).
__device__ __forceinline__ float f8_activation(float g, int gelu)
{
    return f8_activation_steps(
        g, gelu, [](float x) { return __builtin_amdgcn_exp2f(x); }, [](float x) { return __builtin_amdgcn_rcpf(x); });
}

}  // namespace w4a8

// The e4m3 quantization rule (activations and weights alike):
//     amax = max |x| over the block,  s = fl32(amax / 448),
//     code = e4m3(fl32(x / s)), to nearest even
// with IEEE fp32 division.  448 is e4m3's largest value, so the quotient of
// the largest element (at most 448 (1 + 2^-23)) rounds to it and nothing
// saturates.  A block of zeros, or one so small that s would not be a normal
// fp32 number (its reciprocal could overflow), gets s = 0 and zero codes; a
// block that holds a value that is not finite gets s = NaN and zero codes, so
// that every product with it is NaN and no other block is touched.
//
// This header is also compiled for the host by the CPU test suite, which
// checks the corrected quotient against the division for every fp16 input.
#pragma once

#include "quant_rule.h"

namespace w4a8 {

constexpr int kF8Block = 128;
constexpr float kF8Max = 448.0f;

// s of a finite amax >= 0.
W4A8_HD float f8_scale(float amax)
{
    const float s = amax / kF8Max;
    return s < 0x1p-126f ? 0.0f : s;
}

// fl32(x / s) from r = fl32(1 / s): with t = fl32(x r) the residual t s - x is
// exact in one fma, and one step of correction gives the division's result
// for every fp16 x and amax.  In this order of signs a -0 stays -0.
W4A8_HD float f8_quotient(float x, float s, float r)
{
    const float t = x * r;
    return fmaf(-fmaf(t, s, -x), r, t);
}

}  // namespace w4a8

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
// checks the corrected quotient against the division for every fp16 input and
// for the fp32 inputs that come nearest to a border.
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
// taken in one fma, and one step of correction gives the division's result.  In
// this order of signs a -0 stays -0.
//
// That it is the division's result for every fp32 x and s, in steps of the
// quotient: r is within half a step of 1 / s, so t is within 1.5 of x / s, and
// the residual is exact if t is within 1, else off by one unit of the product
// of x's and s's steps.  Before its rounding the corrected value is then off by
// less than 5 / (2 S), S the 24-bit integer of s, and x / s is never nearer
// than 1 / (2 S) to the middle of two steps.  The CPU tests try all pairs that
// lie within 8 / (2 S).  It takes a residual that does not underflow: quotients
// from 2^-11 on (below 2^-10 every e4m3 code is 0, below 1/2 every int8 code)
// with s of at least 2^-90; smaller ones are lifted (f8_reciprocal).
W4A8_HD float f8_quotient(float x, float s, float r)
{
    const float t = x * r;
    return fmaf(-fmaf(t, s, -x), r, t);
}

// What the codes of a block take for its scale s: 0, zero codes, for s = 0 and
// s = NaN; fl32(1 / s); or for s below 2^-90 -fl32(1 / (s 2^64)), whose sign
// says that both sides of the quotient are to be taken 2^64 times as large.
constexpr float kF8Exact = 0x1p-90f, kF8Lift = 0x1p64f;
W4A8_HD float f8_reciprocal(float s)
{
    const float r = 1.0f / (s < kF8Exact ? s * kF8Lift : s);
    return s >= kF8Exact ? r : s > 0.0f ? -r : 0.0f;
}

// silu(g) = g / (1 + e^-g); gelu in its tanh form, 0.5 g (1 + tanh z) =
// g / (1 + e^-2z) with z = sqrt(2 / pi) (g + 0.044715 g^3).
//
// How far from these, with u = 2^-24 (half a step of fp32) and an exponential
// and a reciprocal good to 2 u: the exponent -log2(e) t carries the constant's
// and the product's rounding, 1.3 u of it, for gelu also t's own: four roundings
// in the cubic, two in the factor, 6 u.  As a power it is off by that times |t|,
// and weighs e / (1 + e) in the result.  The sum, the reciprocal, the last
// product and the exponential's own 2 u are another 6 u.  So, of the result,
//     silu  (1.3 |g| w + 6) u,  gelu  (7.3 |t| w + 6) u,  w = 1 / (1 + e^t) <= 1:
// 2^-18.5 for silu at g = -30, 2^-17 for gelu at -5 (t = -16.9) and about half
// of that with half of t; 2^-21 where g > 0.  Far below the rounding of the output
// (2^-11, 2^-4) as long as there is a result: below |g| 2^-126 it may be 0 (e^-g
// overflows to infinity, which gives -0).
template <typename Exp2, typename Rcp>
W4A8_HD float f8_activation_steps(float g, int gelu, Exp2 exp2, Rcp rcp)
{
    float t = g;
    if (gelu)
        t = 1.5957691216057308f * fmaf(0.044715f * g, g * g, g);
    const float e = exp2(-1.4426950408889634f * t);
    return g * rcp(1.0f + e);
}

}  // namespace w4a8

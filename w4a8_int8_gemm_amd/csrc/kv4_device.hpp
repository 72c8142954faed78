// Device pieces shared by the attention kernels over the 4-bit cache: int4
// codes to fp16, cross-lane maxima, and the joining of partial results.
#pragma once

#include <utility>

#include "arrivals.hpp"
#include "device_common.hpp"
#include "kv4.hpp"

namespace w4a8 {

typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Two codes in nibbles 0 and 4 (LO) or 1 and 5 of w to two fp16 values.  With
// its sign bit flipped a nibble is code + 8; or-ed into the low mantissa bits
// of 1024.0 (step 1) it reads 1024 + code + 8, one nibble higher 1024 + 16
// (code + 8).  Both come back exactly, by a subtraction and by a fused
// multiply-add: three packed or bitwise operations for two values, no
// conversion.
__device__ __forceinline__ uint32_t codes_low(uint32_t w)
{
    const uint32_t t = (w & 0x000f000fu) ^ 0x64086408u;
    const h2 r = __builtin_bit_cast(h2, t) + (h2){(_Float16)-1032.0f, (_Float16)-1032.0f};
    return __builtin_bit_cast(uint32_t, r);
}
__device__ __forceinline__ uint32_t codes_high(uint32_t w)
{
    const uint32_t t = (w & 0x00f000f0u) ^ 0x64806480u;
    const h2 r = __builtin_elementwise_fma(__builtin_bit_cast(h2, t), (h2){(_Float16)0.0625f, (_Float16)0.0625f},
                                           (h2){(_Float16)-72.0f, (_Float16)-72.0f});
    return __builtin_bit_cast(uint32_t, r);
}

// The eight codes of a word as an operand, in the order 0 4 1 5 2 6 3 7.
// (Subnormal operands -- the nibble alone in the mantissa, one operation for
// two codes -- are taken exactly, but the matrix unit aligns a sum by the
// operands' exponents, so that their leading zeros cost it up to ten bits.)
__device__ __forceinline__ h8 codes8(uint32_t w)
{
    const uint32_t v = w >> 8;
    const u32x4 r = {codes_low(w), codes_high(w), codes_low(v), codes_high(v)};
    return __builtin_bit_cast(h8, r);
}
// The order above of eight consecutive fp16 values.
__device__ __forceinline__ h8 order8(uint4 x)
{
    const u32x4 r = {__builtin_amdgcn_perm(x.z, x.x, 0x05040100u), __builtin_amdgcn_perm(x.z, x.x, 0x07060302u),
                     __builtin_amdgcn_perm(x.w, x.y, 0x05040100u), __builtin_amdgcn_perm(x.w, x.y, 0x07060302u)};
    return __builtin_bit_cast(h8, r);
}

// Byte g of a and of b in the low bytes of the two halves of a word.
template <int g> __device__ __forceinline__ uint32_t byte_pair(uint32_t a, uint32_t b)
{
    return __builtin_amdgcn_perm(b, a, 0x0c000c00u | ((4u + g) << 16) | g);
}

// Lane N of each row of 16 lanes, in all lanes of the row (folds into the
// instruction that uses it).
template <int N> __device__ __forceinline__ float row_lane(float v)
{
    return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), 0x150 + N, 0xf, 0xf, true));
}

// A table's entry at a uniform address that no kernel writes while this one runs.
__device__ __forceinline__ int scalar_load(const int32_t *p)
{
    return *(const __attribute__((address_space(4))) int32_t *)(uintptr_t)p;
}

// The largest of three; fmaxf would first quieten every operand.
__device__ __forceinline__ float max3(float a, float b, float c)
{
    float r;
    asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
    return r;
}

// Maximum over the lanes up to one's own of 16, and from one's own on; the value of the next lane of 16.
__device__ __forceinline__ uint32_t prefix_max16(uint32_t v)
{
    v = max(v, (uint32_t)W4A8_DPP((int)v, 0x111, 0xf));   // row_shr:1, 2, 4, 8
    v = max(v, (uint32_t)W4A8_DPP((int)v, 0x112, 0xf));
    v = max(v, (uint32_t)W4A8_DPP((int)v, 0x114, 0xf));
    return max(v, (uint32_t)W4A8_DPP((int)v, 0x118, 0xf));
}
__device__ __forceinline__ uint32_t suffix_max16(uint32_t v)
{
    v = max(v, (uint32_t)W4A8_DPP((int)v, 0x101, 0xf));   // row_shl:1, 2, 4, 8
    v = max(v, (uint32_t)W4A8_DPP((int)v, 0x102, 0xf));
    v = max(v, (uint32_t)W4A8_DPP((int)v, 0x104, 0xf));
    return max(v, (uint32_t)W4A8_DPP((int)v, 0x108, 0xf));
}
__device__ __forceinline__ float next_of_16(float v)
{
    return __uint_as_float((uint32_t)W4A8_DPP((int)__float_as_uint(v), 0x12f, 0xf));   // row_ror:15
}

// The least of exponents over -128 over groups of lanes.
template <int width> __device__ __forceinline__ int group_min_exponent(int e)
{
    return 128 - (int)group_max_u32<width>((uint32_t)(128 - e));
}

// Sum over groups of lanes, and the sum over the lanes up to and with one's own.
template <int width> __device__ __forceinline__ uint32_t group_sum_u32(uint32_t v)
{
    return lane_reduce<width>(v, [](uint32_t a, uint32_t b) { return a + b; });
}
__device__ __forceinline__ int64_t wave_sum64(int64_t v)
{
#pragma unroll
    for (int i = 32; i; i >>= 1)
        v += __shfl_xor(v, i);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)v), hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(v >> 32));
    return (int64_t)(((uint64_t)hi << 32) | lo);
}
__device__ __forceinline__ int prefix_sum(int v)
{
    v += W4A8_DPP(v, 0x111, 0xf);                    // row_shr:1, 2, 4, 8
    v += W4A8_DPP(v, 0x112, 0xf);
    v += W4A8_DPP(v, 0x114, 0xf);
    v += W4A8_DPP(v, 0x118, 0xf);
    v += W4A8_DPP(v, 0x142, 0xa);                    // row_bcast:15 into rows 1, 3
    v += W4A8_DPP(v, 0x143, 0xc);                    // row_bcast:31 into rows 2, 3
    return v;
}

// f(0), ..., f(N - 1) with the index as a constant.
template <int N, typename F, int... I>
__device__ __forceinline__ void each_of(F &&f, std::integer_sequence<int, I...>)
{
    (f(std::integral_constant<int, I>()), ...);
}
template <int N, typename F> __device__ __forceinline__ void each(F &&f)
{
    each_of<N>(f, std::make_integer_sequence<int, N>());
}

// Maximum of `and_` and v over the lanes l, l ^ 16, l ^ 32, l ^ 48; of v over l, l ^ 32.
__device__ __forceinline__ float max_rows(float v, float and_)
{
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    const uint32_t m = __float_as_uint(max3(__uint_as_float(r[0]), __uint_as_float(r[1]), __uint_as_float(r[1])));
    const auto q = __builtin_amdgcn_permlane32_swap(m, m, false, false);
    return max3(__uint_as_float(q[0]), __uint_as_float(q[1]), and_);
}
__device__ __forceinline__ float max_halves(float v)
{
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return max3(__uint_as_float(r[0]), __uint_as_float(r[1]), __uint_as_float(r[1]));
}
// The same of unsigned values.
__device__ __forceinline__ uint32_t max_rows_u32(uint32_t v)
{
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    const uint32_t m = max(r[0], r[1]);
    const auto q = __builtin_amdgcn_permlane32_swap(m, m, false, false);
    return max(q[0], q[1]);
}
__device__ __forceinline__ uint32_t max_halves_u32(uint32_t v)
{
    const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return max(r[0], r[1]);
}
__device__ __forceinline__ float sum_halves(float v)
{
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ float sum_rows(float v)
{
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return sum_halves(__uint_as_float(r[0]) + __uint_as_float(r[1]));
}

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

// A scale's bits without its sign (abs_bits): numbers in their order, what is not finite
// above them.  The exponent floor(log2 v) of a finite one, -127 for 0.
constexpr uint32_t kNotFinite = 0x7f800000u;
__device__ __forceinline__ int exponent_of(uint32_t bits) { return (int)(bits >> 23) - 127; }

// Weights p = 2^(score - ref) are multiplied with their value's scale and
// rounded to fp16.  The reference is not the running maximum but follows it
// where a weight could leave fp16's range: for scales below 2^(e + 1) a score
// above `bound` = ref + kRange - e.  Then ref = (the row's largest score) + e -
// kHeadroom, so that its weight times the largest scale is about 2^kHeadroom:
// products stay below 2^(kRange + 1), and those 26 binades under the largest
// keep all their bits (a row's heaviest key may have a code of 0 in some
// element, whose result then comes from light keys alone; 7 binades of
// headroom were too few there).  Sum and output have the same reference, and
// any gives the same quotient.  e is a row's own, from the scales of the keys
// that it sees: another's may be anything.  An unseen key's weight is 0, but 0
// times a scale that is not finite is not: such scales are taken out of the
// products, and rows that see one get NaN in the elements of its group.
constexpr int kHeadroom = 12, kRange = 14;
// The kernel for few rows takes weights as two fp16 values where a row sees at most this many keys.
constexpr int kFewKeys = 1024;
constexpr float kFarBelow = -3.4028234664e38f; // reference before any key: under every score
// Exponent of the largest scale before any key, and the least that is told
// apart: smaller scales' values round to 0 in fp16 (8 * 2^-40 < 2^-25) and
// are taken as that, and weights stay below 2^55, sums of 2^30 of them in range.
constexpr int kNoScale = -40;
// The reference for a row whose largest score is m (it never falls), and the
// bound above one.  Scores from 2^24 on are held in steps of 2 and more: where a
// sum is off by more than a binade the reference is m itself, and where the
// bound would be up by more than half a one it is the reference.
__device__ __forceinline__ float reference_for(float ref, float m, int e)
{
    const float below = (float)(kHeadroom - e), next = m - below;
    return fmaxf(ref, fabsf((m - next) - below) > 1.0f ? m : next);
}
__device__ __forceinline__ float bound_for(float ref, int e)
{
    const float above = (float)(kRange - e), bound = ref + above;
    return (bound - ref) - above > 0.5f ? ref : bound;
}
__device__ __forceinline__ uint32_t cap_of(int e) { return (uint32_t)(e + 128) << 23; }   // bits of 2^(e + 1)

// Where parts of a result that several workgroups compute meet.
struct Partial {
    float *base;                // [slots][slot_rows * (D + 2)]: output, reference and sum
    int slots, slot_rows;
    uint64_t *counters;         // [items][kCounterStride]
    int grid;
    int row_limit;              // rows a kv head: the most for the kernel of few rows, one less for the other
    uint32_t over_group;        // division of a row by the group, see query_of()
};

// Row = query * group + head of the group.  The quotient of rows < 2^16 by
// ceil(2^32 / group) is exact; one query head a kv head needs no division.
inline uint32_t over_group(int group) { return (uint32_t)(((uint64_t(1) << 32) + group - 1) / group); }
__device__ __forceinline__ int query_of(uint32_t row, uint32_t over, int group)
{
    return group == 1 ? (int)row : row < 65536u ? (int)__umulhi(row, over) : (int)(row / (uint32_t)group);
}

}  // namespace w4a8

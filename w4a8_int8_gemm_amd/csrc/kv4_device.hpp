// Device pieces shared by the attention kernels over the 4-bit cache: int4
// codes to fp16, cross-lane maxima, and the joining of partial results.
#pragma once

#include <utility>

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

// A value that is the same in all lanes, as a scalar.
__device__ __forceinline__ int64_t uniform(int64_t v)
{
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)v), hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(v >> 32));
    return (int64_t)(((uint64_t)hi << 32) | lo);
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

// Maximum over the lanes l, l ^ 32, and over l, l ^ 16, l ^ 32, l ^ 48.
__device__ __forceinline__ float max_halves(float v)
{
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float max_rows(float v)
{
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return max_halves(fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1])));
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

// The exponent floor(log2 v) of the largest scale of a step, -127 for 0.
__device__ __forceinline__ int exponent_of(float v) { return (int)(__float_as_uint(v) >> 23) - 127; }

// The weights p = exp2(s - ref) times a value's scale have to fit fp16, whose
// normal numbers span 30 binades.  ref = (largest score seen) + (exponent of
// the largest scale seen) - kHeadroom puts every weight below 2^14 and lets
// scores times scales 28 binades under the largest keep all their bits; any
// reference gives the same quotient, so sum and output need no correction.
constexpr int kHeadroom = 13;
constexpr int kNoScale = -100;                // exponent before any key

// Values that other workgroups, on other chiplets with L2 caches of their
// own, wrote or will read within one launch: loads and stores at device scope.
__device__ __forceinline__ void store_shared(float *p, float a, float b)
{
    const uint64_t v = ((uint64_t)__float_as_uint(b) << 32) | __float_as_uint(a);
    __hip_atomic_store(reinterpret_cast<uint64_t *>(p), v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float2 load_shared(const float *p)
{
    const uint64_t v = __hip_atomic_load(reinterpret_cast<const uint64_t *>(p), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    return make_float2(__uint_as_float((uint32_t)v), __uint_as_float((uint32_t)(v >> 32)));
}

// Counts the arrivals at one counter of this call: true for the last of
// `parts`.  The counter's upper 48 bits name the call and its lower 16 count;
// one that carries another call's tag counts as zero, so nothing has to be
// cleared before the call, and the last arrival clears it, so that a captured
// call can run again.  The caller's stores are complete before (all waves
// have waited for theirs).
__device__ __forceinline__ bool arrive_last(uint64_t *counter, uint64_t tag, int parts)
{
    uint64_t seen = __hip_atomic_load(counter, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    for (;;) {
        const uint64_t base = (seen & ~uint64_t(0xffff)) == tag ? seen : tag;
        const bool last = (int)(base & 0xffff) == parts - 1;
        const uint64_t next = last ? 0 : base + 1;
        if (__hip_atomic_compare_exchange_strong(counter, &seen, next, __ATOMIC_RELAXED, __ATOMIC_RELAXED,
                                                 __HIP_MEMORY_SCOPE_AGENT))
            return last;
    }
}

}  // namespace w4a8

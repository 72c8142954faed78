// Where workgroups of one launch meet in a workspace: stores and loads at
// device scope, and counters that need no clearing (gfx950).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace w4a8 {

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

// Arrivals at one counter of this call, without anything to clear before it:
// the upper 48 bits name the call, the lower 16 count.  announce(), by every
// workgroup before its arrival, gives a counter with another call's tag this
// call's, once (the exchange fails for all but the first); arrive() then is
// one addition, true for the last of `parts`, which clears the counter, so
// that a captured call can run again.  (One exchange per arrival instead of
// the addition would be tried again by all that lose it: 64 workgroups took
// 100 us.)  The caller's stores are complete before arrive().
__device__ __forceinline__ void announce(uint64_t *counter, uint64_t tag)
{
    uint64_t seen = __hip_atomic_load(counter, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if ((seen & ~uint64_t(0xffff)) != tag)
        __hip_atomic_compare_exchange_strong(counter, &seen, tag, __ATOMIC_RELAXED, __ATOMIC_RELAXED,
                                             __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ bool arrive(uint64_t *counter, int parts)
{
    const uint64_t n = __hip_atomic_fetch_add(counter, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) & 0xffff;
    if ((int)n != parts - 1)
        return false;
    __hip_atomic_store(counter, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    return true;
}

}  // namespace w4a8

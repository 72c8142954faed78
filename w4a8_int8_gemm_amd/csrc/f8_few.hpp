// How the products of few tokens are laid out over the chip (host side).
#pragma once

#include "f8.hpp"
#include "kv4.hpp"

#ifndef F8_FEW_LDS
#define F8_FEW_LDS (72 * 1024)
#endif

namespace w4a8 {

constexpr int kF8FewTokens = 64;               // four blocks of 16

struct F8Few {
    int blocks;                 // blocks of 16 columns a workgroup: 1 or 2
    int splits;                 // ranges of K
    uint64_t tag;               // of the call among the counters
    uint64_t *counters;         // one for each 128 columns, kCounterStride apart
    float *sums;
};

inline size_t f8_few_counter_bytes(int64_t N) { return kv4_counter_bytes((N + 127) / 128, 1); }

inline F8Few f8_few_plan(int64_t M, int64_t N, int64_t K, bool gated, bool quantize)
{
    (void)M; (void)K; (void)quantize;
    F8Few f{};
    const int64_t chunks = (N + 15) / 16;
    f.blocks = chunks >= (gated ? 768 : 1024) ? 2 : 1;
    f.splits = 1;
    return f;
}

inline size_t f8_few_workspace(int64_t M, int64_t N, int64_t K, bool gated, bool quantize)
{
    const F8Few f = f8_few_plan(M, N, K, gated, quantize);
    if (f.splits == 1 && !quantize)
        return 0;
    const int sides = gated && f.splits > 1 ? 2 : 1;
    return f8_few_counter_bytes(N) + (size_t)((N + 127) / 128) * f.splits * sides * (size_t)M * 128 * sizeof(float);
}

}  // namespace w4a8

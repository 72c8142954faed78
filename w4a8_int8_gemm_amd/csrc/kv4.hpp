// The 4-bit key/value cache as the kernels see it, and launchers of the
// operators around it (include/w4a8.h gives formats and formulas).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.hpp"
#include "kv4_index.h"

namespace w4a8 {

// Checked by the C entry points; shift = log2(page_size).
struct Kv4Cache {
    uint8_t *k, *v;             // [pages, heads, 1 << shift, D / 2], rows stored transposed
    float *ks, *vs;             // [pages, heads, 1 << shift, D / G]
    int64_t pages;
    int heads, shift, D, G;

    // Row of a page's token for one head, in rows of the four arrays.
    __host__ __device__ int64_t row(int64_t page, int head, int at) const
    {
        return ((page * heads + head) << shift) + at;
    }
};

struct Kv4AttnArgs {
    const uint16_t *q;          // [T, q_heads, D], token stride q_stride
    int64_t q_stride, T;
    int q_heads, group;         // group = q_heads / kv heads
    const int32_t *table;       // [B, max_pages]
    int max_pages;
    const int32_t *kv_lens;     // [B]
    const int32_t *q_starts;    // [B + 1] or null (one query a sequence)
    int B;
    int max_q;
    bool causal;
    int window;                 // 0: none
    float scale;
    uint16_t *out;              // [T, q_heads, D]
    float *lse;                 // [T, q_heads] or null
    void *workspace;
    uint64_t tag;               // of this call among the counters in the workspace
};

void launch_rotary(const uint16_t *x, int64_t x_stride, const int64_t *pos, const float *inv_freq,
                   int64_t T, int heads, int D, int R, int axes, const int *sections,
                   bool interleaved, uint16_t *out, int64_t out_stride, hipStream_t st);

void launch_kv4_write(const uint16_t *k, int64_t k_stride, const uint16_t *v, int64_t v_stride,
                      const int64_t *slots, int64_t T, const Kv4Cache &c, hipStream_t st);
void launch_kv4_read(const Kv4Cache &c, const int64_t *slots, int64_t T, uint16_t *k, uint16_t *v,
                     hipStream_t st);

size_t kv4_attention_workspace(int q_heads, int kv_heads, int D, int64_t T, int B, int max_q);
// Whether the call's workgroups (of 256 threads) stay under the 2^32 threads of a launch, past which it
// would wrap without an error.
bool kv4_attention_fits(const Kv4Cache &c, const Kv4AttnArgs &a);
void launch_kv4_attention(const Kv4Cache &c, const Kv4AttnArgs &a, hipStream_t st);

// Sequences of at most this many query rows a kv head (queries x query heads):
// two blocks of 16.  Four blocks against the other kernel's tile of 128: short
// sequences are faster there (11 of up to 71 tokens, 13 queries x 8 heads: 25 us
// with four, 15.7 without), long ones a little slower (2 x 14 queries x 4 heads
// behind 4625 keys: 39 us with four, 43 without).
constexpr int kDecodeRows = 32;
// A counter for each (sequence, head), on lines of their own: arrivals on one line queue up.
constexpr int kCounterStride = 16;
inline size_t kv4_counter_bytes(int64_t B, int heads) { return ((size_t)B * heads * kCounterStride * 8 + 255) & ~size_t(255); }
void launch_kv4_decode(const Kv4Cache &c, const Kv4AttnArgs &a, int rows, hipStream_t st);
// The other sequences, those with more than row_limit rows a kv head.
void launch_kv4_prefill(const Kv4Cache &c, const Kv4AttnArgs &a, int row_limit, void *workspace, hipStream_t st);

// Sequence b of the call.
__device__ __forceinline__ Kv4Seq kv4_sequence(const Kv4AttnArgs &a, int shift, int b)
{
    const int start = a.q_starts ? a.q_starts[b] : b;
    const int end = a.q_starts ? a.q_starts[b + 1] : b + 1;
    return kv4_cut(start, end, a.kv_lens[b], (int)a.T, a.max_q, a.max_pages << shift);
}

}  // namespace w4a8

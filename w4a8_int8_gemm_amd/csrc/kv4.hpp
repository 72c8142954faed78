// The 4-bit key/value cache as the kernels see it, and launchers of the
// operators around it (include/w4a8.h gives formats and formulas).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.hpp"

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
    int64_t B;
    int max_q;
    bool causal;
    int window;                 // 0: none
    float scale;
    uint16_t *out;              // [T, q_heads, D]
    float *lse;                 // [T, q_heads] or null
    void *workspace;
    int num_cu;
};

void launch_rotary(const uint16_t *x, int64_t x_stride, const int64_t *pos, const float *inv_freq,
                   int64_t T, int heads, int D, int R, int axes, const int *sections,
                   bool interleaved, uint16_t *out, int64_t out_stride, hipStream_t st);

void launch_kv4_write(const uint16_t *k, int64_t k_stride, const uint16_t *v, int64_t v_stride,
                      const int64_t *slots, int64_t T, const Kv4Cache &c, hipStream_t st);
void launch_kv4_read(const Kv4Cache &c, const int64_t *slots, int64_t T, uint16_t *k, uint16_t *v,
                     hipStream_t st);

size_t kv4_attention_workspace(int q_heads, int kv_heads, int D, int64_t T, int64_t B, int max_q);
void launch_kv4_attention(const Kv4Cache &c, const Kv4AttnArgs &a, hipStream_t st);

// A sequence's queries and keys as the device-side tables give them, cut to
// what the call's buffers hold.
struct Kv4Seq {
    int64_t q0;                 // first query row
    int m;                      // queries
    int64_t n;                  // keys
};
__device__ __forceinline__ Kv4Seq kv4_sequence(const Kv4AttnArgs &a, int shift, int64_t b)
{
    Kv4Seq s;
    const int64_t most = (int64_t)a.max_pages << shift;
    const int64_t n = a.kv_lens[b];
    s.n = n < 0 ? 0 : n < most ? n : most;
    if (a.q_starts) {
        const int64_t q0 = a.q_starts[b], q1 = a.q_starts[b + 1];
        s.q0 = q0 < 0 ? 0 : q0;
        const int64_t end = q1 < a.T ? q1 : a.T;
        int64_t m = end - s.q0;
        m = m < 0 ? 0 : m;
        s.m = (int)(m < a.max_q ? m : a.max_q);
    } else {
        s.q0 = b;
        s.m = b < a.T ? 1 : 0;
    }
    return s;
}

// The keys query i of m sees: [lo, hi).
__device__ __forceinline__ void kv4_visible(const Kv4AttnArgs &a, int64_t n, int m, int i,
                                            int64_t &lo, int64_t &hi)
{
    lo = 0;
    hi = n;
    if (a.causal) {
        hi = n - m + i + 1;
        if (a.window > 0 && hi - a.window > 0)
            lo = hi - a.window;
        hi = hi < 0 ? 0 : hi;
    }
}

}  // namespace w4a8

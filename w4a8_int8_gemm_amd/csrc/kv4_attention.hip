// Attention over the 4-bit paged cache (include/w4a8.h: kv4_attention).
//
// One wavefront per (query row, query head): each lane scores one key of a
// step of 64, the running maximum and sum of the softmax are kept over the
// steps, and the lanes then hold the output's elements.
#include "kv4_device.hpp"

namespace w4a8 {

namespace {

__device__ __forceinline__ float wave_max(float v)
{
    for (int i = 32; i; i >>= 1)
        v = fmaxf(v, __shfl_xor(v, i));
    return v;
}
__device__ __forceinline__ float wave_sum(float v)
{
    for (int i = 32; i; i >>= 1)
        v += __shfl_xor(v, i);
    return v;
}

__device__ __forceinline__ float nibble(uint32_t word, int e)
{
    return (float)((int32_t)(word << (28 - 4 * e)) >> 28);
}

// grid.x over the rows (sequence, query index), grid.y over the query heads / 4.
__global__ __launch_bounds__(256) void kv4_attention_kernel(Kv4Cache c, Kv4AttnArgs a, int row_limit)
{
    __shared__ float qs[4][256], ps[4][64];
    __shared__ int64_t rows[4][64];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int b = blockIdx.x / a.max_q;
    const int i = (int)(blockIdx.x % a.max_q);
    const int h = blockIdx.y * 4 + wave;
    const Kv4Seq s = kv4_sequence(a, c.shift, b);
    const bool active = i < s.m && h < a.q_heads;
    if ((int64_t)s.m * a.group <= row_limit)
        return;
    const int lo = kv4_lo(s.n, s.m, i, a.window), hi = kv4_hi(s.n, s.m, i, a.causal);
    const int D = c.D, n32 = D / 32, NG = D / c.G;
    const int64_t qrow = s.q0 + i;
    const int hk = active ? h / a.group : 0;
    if (active)
        for (int d = lane; d < D; d += 64)
            qs[wave][d] = h2f(a.q[qrow * a.q_stride + (int64_t)h * D + d]);
    float m = -INFINITY, l = 0.0f, o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    const int64_t steps = ((int64_t)s.n + 63) / 64;
    for (int64_t st = lo / 64; st < steps; ++st) {
        __syncthreads();
        const int64_t j = st * 64 + lane;
        bool seen = active && j >= lo && j < hi;
        int64_t row = 0;
        if (seen) {
            const int64_t page = a.table[(int64_t)b * a.max_pages + (j >> c.shift)];
            seen = page >= 0 && page < c.pages;
            if (seen)
                row = c.row(page, hk, (int)(j & ((1 << c.shift) - 1)));
        }
        float x = -INFINITY;
        if (seen) {
            x = 0.0f;
            for (int g = 0; g < NG; ++g) {
                float acc = 0.0f;
                for (int w = g * c.G / 8; w < (g + 1) * c.G / 8; ++w) {
                    const uint32_t word = *reinterpret_cast<const uint32_t *>(
                        c.k + row * (D / 2) + ((w % 4) * n32 + w / 4) * 4);
                    for (int e = 0; e < 8; ++e)
                        acc = fmaf(qs[wave][w * 8 + e], nibble(word, e), acc);
                }
                x = fmaf(acc, c.ks[row * NG + g], x);
            }
            x *= a.scale * kLog2e;
        }
        const float top = fmaxf(m, wave_max(x));
        const float ref = top == -INFINITY ? 0.0f : top;
        const float alpha = m == -INFINITY ? 0.0f : exp2f(m - ref);
        const float p = seen ? exp2f(x - ref) : 0.0f;
        m = top;
        l = fmaf(l, alpha, wave_sum(p));
        for (int e = 0; e < 4; ++e)
            o[e] *= alpha;
        ps[wave][lane] = p;
        rows[wave][lane] = seen ? row : -1;
        __syncthreads();
        for (int jj = 0; jj < 64; ++jj) {
            const int64_t r = rows[wave][jj];
            if (r < 0)
                continue;
            const float pj = ps[wave][jj];
            for (int e = 0; e < D / 64; ++e) {
                const int d = lane + 64 * e, byte = d / 2;
                const uint8_t u = c.v[r * (D / 2) + (byte % 16) * n32 + byte / 16];
                o[e] = fmaf(pj * c.vs[r * NG + d / c.G], nibble(u, d & 1), o[e]);
            }
        }
    }
    if (!active)
        return;
    for (int e = 0; e < D / 64; ++e)
        a.out[(qrow * a.q_heads + h) * D + lane + 64 * e] = f2h(l > 0.0f ? o[e] / l : 0.0f);
    if (a.lse && lane == 0)
        a.lse[qrow * a.q_heads + h] = l > 0.0f ? (m + log2f(l)) * kLn2 : -INFINITY;
}

}  // namespace

namespace {

// Rows a kv head that the kernel for few rows is launched for: what a sequence
// can have, or that kernel's limit.
int decode_rows(int D, int group, int64_t max_q)
{
    const int limit = kv4_decode_limit(D);
    return group * max_q < limit ? (int)(group * max_q) : limit;
}

}  // namespace

size_t kv4_attention_workspace(int q_heads, int kv_heads, int D, int64_t T, int B, int max_q)
{
    const int rows = decode_rows(D, q_heads / kv_heads, max_q < T ? max_q : T);
    return kv4_counter_bytes(B, kv_heads) + (size_t)(B * (int64_t)kv_heads + kPartsMore) * rows * (D + 2) * sizeof(float);
}

void launch_kv4_attention(const Kv4Cache &c, const Kv4AttnArgs &a, hipStream_t st)
{
    const int limit = kv4_decode_limit(c.D);
    if (a.group <= limit)
        launch_kv4_decode(c, a, decode_rows(c.D, a.group, a.max_q), st);
    if ((int64_t)a.group * a.max_q > limit)
        hipLaunchKernelGGL(kv4_attention_kernel, dim3((unsigned)((int64_t)a.B * a.max_q), (unsigned)((a.q_heads + 3) / 4)),
                           dim3(256), 0, st, c, a, a.group <= limit ? limit : 0);
}

}  // namespace w4a8

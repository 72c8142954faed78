// Writing keys and values into the 4-bit paged cache and reading them back
// (include/w4a8.h: kv4_write, kv4_read).
//
// Both are bound by HBM: the writer reads 2 bytes and writes 1/2 (+ 4 / G) per
// element, the reader the other way round.
//
// Four neighbouring lanes have a (token, head) row of K or V, lane b the
// elements 32 g + 8 b ..+7 of every 32: 16 bytes of fp16 for each g, and in
// the cache, whose rows are stored transposed, D / 8 bytes in one run (K's
// words b n .. b n + n - 1; V's bytes 4 b n .. 4 b n + 4 n - 1, after a
// transposition of 4 x 4 bytes in registers).  A scale's maximum is taken over
// a lane's own elements and the four lanes.  Measured at 8 heads of 128: reading
// 65533 tokens (G = 32, 353 MB) 77 us, 4.6 TB/s; 4516 tokens (G = 64, 23.7 MB)
// written in 9.2 us and read in 7.2 us, half the rate of the long read.
#include "kv4.hpp"

namespace w4a8 {

namespace {

// Eight codes (bytes, k = 0..7) to eight nibbles, element 0 lowest.
__device__ __forceinline__ uint32_t pack_nibbles(uint2 c)
{
    const uint32_t a = c.x & 0x0f0f0f0fu, b = c.y & 0x0f0f0f0fu;
    const uint32_t x = a | (a >> 4), y = b | (b >> 4);            // bytes 0 and 2 hold pairs
    return (x & 0xffu) | ((x >> 8) & 0xff00u) | ((y & 0xffu) << 16) | ((y << 8) & 0xff000000u);
}

// Byte i of word j becomes byte j of word i.
__device__ __forceinline__ void transpose4(uint32_t (&w)[4])
{
    const uint32_t a = __builtin_amdgcn_perm(w[1], w[0], 0x05010400u), b = __builtin_amdgcn_perm(w[1], w[0], 0x07030602u);
    const uint32_t c = __builtin_amdgcn_perm(w[3], w[2], 0x05010400u), d = __builtin_amdgcn_perm(w[3], w[2], 0x07030602u);
    w[0] = __builtin_amdgcn_perm(c, a, 0x05040100u);
    w[1] = __builtin_amdgcn_perm(c, a, 0x07060302u);
    w[2] = __builtin_amdgcn_perm(d, b, 0x05040100u);
    w[3] = __builtin_amdgcn_perm(d, b, 0x07060302u);
}

// A lane's natural words (word g: elements 32 g + 8 b ..+7) of a V row to its
// stored ones, whose bytes run over g first; and back.
template <int N> __device__ __forceinline__ void v_stored(uint32_t (&w)[N])
{
    if constexpr (N == 2) {
        const uint32_t a = w[0], b = w[1];
        w[0] = __builtin_amdgcn_perm(b, a, 0x05010400u);
        w[1] = __builtin_amdgcn_perm(b, a, 0x07030602u);
    } else if constexpr (N == 4) {
        transpose4(w);
    } else {
        uint32_t a[4] = {w[0], w[1], w[2], w[3]}, b[4] = {w[4], w[5], w[6], w[7]};
        transpose4(a);
        transpose4(b);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            w[2 * e] = a[e], w[2 * e + 1] = b[e];
    }
}
template <int N> __device__ __forceinline__ void v_natural(uint32_t (&w)[N])
{
    if constexpr (N == 2) {
        const uint32_t a = w[0], b = w[1];
        w[0] = __builtin_amdgcn_perm(b, a, 0x06040200u);
        w[1] = __builtin_amdgcn_perm(b, a, 0x07050301u);
    } else if constexpr (N == 4) {
        transpose4(w);
    } else {
        uint32_t a[4] = {w[0], w[2], w[4], w[6]}, b[4] = {w[1], w[3], w[5], w[7]};
        transpose4(a);
        transpose4(b);
#pragma unroll
        for (int g = 0; g < 4; ++g)
            w[g] = a[g], w[4 + g] = b[g];
    }
}

template <int N> __device__ __forceinline__ void store_words(uint8_t *p, const uint32_t (&w)[N])
{
    if constexpr (N == 2) {
        *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
        for (int i = 0; i < N / 4; ++i)
            reinterpret_cast<uint4 *>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    }
}
template <int N> __device__ __forceinline__ void load_words(uint32_t (&w)[N], const uint8_t *p)
{
    if constexpr (N == 2) {
        const uint2 x = *reinterpret_cast<const uint2 *>(p);
        w[0] = x.x, w[1] = x.y;
    } else {
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            const uint4 x = reinterpret_cast<const uint4 *>(p)[i];
            w[4 * i] = x.x, w[4 * i + 1] = x.y, w[4 * i + 2] = x.z, w[4 * i + 3] = x.w;
        }
    }
}

// grid.y: K, V
template <int D, int NG>
__global__ __launch_bounds__(256) void kv4_write_kernel(const uint16_t *__restrict__ k, int64_t k_stride,
                                                        const uint16_t *__restrict__ v, int64_t v_stride,
                                                        const int64_t *__restrict__ slots, int64_t T, Kv4Cache c)
{
    constexpr int N = D / 32, PER = N / NG;
    const uint32_t i = blockIdx.x * 256u + threadIdx.x, row_of = i >> 2, b = i & 3;
    const int64_t t = row_of / (uint32_t)c.heads;
    const int head = row_of % (uint32_t)c.heads;
    if (t >= T)                                          // whole groups of four lanes
        return;
    const bool is_v = blockIdx.y != 0;
    const uint16_t *src = (is_v ? v + t * v_stride : k + t * k_stride) + head * D + 8 * b;
    uint4 x[N];
#pragma unroll
    for (int g = 0; g < N; ++g)
        x[g] = load_nt(reinterpret_cast<const uint4 *>(src + 32 * g));
    const int64_t slot = slots[t];
    if (slot < 0 || slot >= (c.pages << c.shift))
        return;
    float s[NG];
    uint32_t w[N];
#pragma unroll
    for (int q = 0; q < NG; ++q) {
        uint32_t m = 0;
#pragma unroll
        for (int g = q * PER; g < (q + 1) * PER; ++g)
            m = max(m, absmax_bits8(x[g]));
        s[q] = quant_scale(h2f((uint16_t)group_max_u32<4>(m)), 7.0f);
        const float r = 1.0f / s[q];
#pragma unroll
        for (int g = q * PER; g < (q + 1) * PER; ++g)
            w[g] = pack_nibbles(quant_chunk8(x[g], s[q], r, 7.0f));
    }
    if (is_v)
        v_stored(w);
    const int64_t row = c.row(slot >> c.shift, head, (int)(slot & ((1 << c.shift) - 1)));
    store_words(((is_v ? c.v : c.k) + row * (D / 2)) + b * (D / 8), w);
    float *sp = (is_v ? c.vs : c.ks) + row * NG;
#pragma unroll
    for (int q = 0; q < NG; ++q)
        if (b == q)
            sp[q] = s[q];
}

// grid.y: K, V
template <int D, int NG>
__global__ __launch_bounds__(256) void kv4_read_kernel(Kv4Cache c, const int64_t *__restrict__ slots, int64_t T,
                                                       uint16_t *__restrict__ k, uint16_t *__restrict__ v)
{
    constexpr int N = D / 32, PER = N / NG;
    const uint32_t i = blockIdx.x * 256u + threadIdx.x, row_of = i >> 2, b = i & 3;
    const int64_t t = row_of / (uint32_t)c.heads;
    const int head = row_of % (uint32_t)c.heads;
    if (t >= T)
        return;
    const bool is_v = blockIdx.y != 0;
    const int64_t slot = slots[t];
    const bool there = slot >= 0 && slot < (c.pages << c.shift);
    uint32_t w[N];
    float s[NG];
    if (there) {
        const int64_t row = c.row(slot >> c.shift, head, (int)(slot & ((1 << c.shift) - 1)));
        load_words(w, (is_v ? c.v : c.k) + row * (D / 2) + b * (D / 8));
        const float *sp = (is_v ? c.vs : c.ks) + row * NG;
#pragma unroll
        for (int q = 0; q < NG; ++q)
            s[q] = sp[q];
    } else {
#pragma unroll
        for (int g = 0; g < N; ++g)
            w[g] = 0;
#pragma unroll
        for (int q = 0; q < NG; ++q)
            s[q] = 0.0f;
    }
    if (is_v)
        v_natural(w);
    uint16_t *dst = (is_v ? v : k) + (int64_t)row_of * D + 8 * b;
#pragma unroll
    for (int g = 0; g < N; ++g) {
        float f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            f[e] = (float)((int32_t)(w[g] << (28 - 4 * e)) >> 28) * s[g / PER];
        *reinterpret_cast<uint4 *>(dst + 32 * g) =
            make_uint4(pack_h2(f[0], f[1]), pack_h2(f[2], f[3]), pack_h2(f[4], f[5]), pack_h2(f[6], f[7]));
    }
}

template <typename F> void each_geometry(const Kv4Cache &c, F &&f)
{
    switch (c.D * 8 + c.D / c.G) {
    case 64 * 8 + 1: f(std::integral_constant<int, 64>(), std::integral_constant<int, 1>()); return;
    case 64 * 8 + 2: f(std::integral_constant<int, 64>(), std::integral_constant<int, 2>()); return;
    case 128 * 8 + 1: f(std::integral_constant<int, 128>(), std::integral_constant<int, 1>()); return;
    case 128 * 8 + 2: f(std::integral_constant<int, 128>(), std::integral_constant<int, 2>()); return;
    case 128 * 8 + 4: f(std::integral_constant<int, 128>(), std::integral_constant<int, 4>()); return;
    case 256 * 8 + 1: f(std::integral_constant<int, 256>(), std::integral_constant<int, 1>()); return;
    case 256 * 8 + 2: f(std::integral_constant<int, 256>(), std::integral_constant<int, 2>()); return;
    default: f(std::integral_constant<int, 256>(), std::integral_constant<int, 4>()); return;
    }
}

}  // namespace

void launch_kv4_write(const uint16_t *k, int64_t k_stride, const uint16_t *v, int64_t v_stride,
                      const int64_t *slots, int64_t T, const Kv4Cache &c, hipStream_t st)
{
    const dim3 grid((unsigned)((T * c.heads * 4 + 255) / 256), 2);
    each_geometry(c, [&](auto d, auto ng) {
        hipLaunchKernelGGL((kv4_write_kernel<decltype(d)::value, decltype(ng)::value>), grid, dim3(256), 0, st, k, k_stride,
                           v, v_stride, slots, T, c);
    });
}

void launch_kv4_read(const Kv4Cache &c, const int64_t *slots, int64_t T, uint16_t *k, uint16_t *v, hipStream_t st)
{
    const dim3 grid((unsigned)((T * c.heads * 4 + 255) / 256), 2);
    each_geometry(c, [&](auto d, auto ng) {
        hipLaunchKernelGGL((kv4_read_kernel<decltype(d)::value, decltype(ng)::value>), grid, dim3(256), 0, st, c, slots, T, k,
                           v);
    });
}

}  // namespace w4a8

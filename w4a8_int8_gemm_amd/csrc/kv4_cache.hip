// Writing keys and values into the 4-bit paged cache and reading them back
// (include/w4a8.h: kv4_write, kv4_read).
//
// Both are bound by HBM: the writer reads 2 bytes and writes 1/2 (+ 4 / G) per
// element, the reader the other way round.
#include "kv4.hpp"

namespace w4a8 {

namespace {

// Maximum over groups of W consecutive lanes (4, 8, 16 or 32).
template <int W>
__device__ __forceinline__ uint32_t scale_group_max(uint32_t v)
{
    if constexpr (W == 32) {
        v = group_max_u32<16>(v);
        return max(v, (uint32_t)__shfl_xor((int)v, 16));
    } else {
        return group_max_u32<W>(v);
    }
}

// Eight codes (bytes, k = 0..7) to eight nibbles, element 0 lowest.
__device__ __forceinline__ uint32_t pack_nibbles(uint2 c)
{
    const uint32_t a = c.x & 0x0f0f0f0fu, b = c.y & 0x0f0f0f0fu;
    const uint32_t x = a | (a >> 4), y = b | (b >> 4);            // bytes 0 and 2 hold pairs
    return (x & 0xffu) | ((x >> 8) & 0xff00u) | ((y & 0xffu) << 16) | ((y << 8) & 0xff000000u);
}

// One lane per 8 elements of a (token, head) row; G / 8 neighbouring lanes share a scale.
template <int G>
__global__ __launch_bounds__(256) void kv4_write_kernel(const uint16_t *__restrict__ k,
                                                        int64_t k_stride,
                                                        const uint16_t *__restrict__ v,
                                                        int64_t v_stride,
                                                        const int64_t *__restrict__ slots,
                                                        int64_t T, Kv4Cache c)
{
    const int per = c.D / 8, n = c.D / 32;
    const int64_t work = T * c.heads * per;
    const int64_t w = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const bool inside = w < work;
    const int64_t wc = inside ? w : work - 1;
    const int chunk = (int)(wc % per);
    const int64_t th = wc / per;
    const int head = (int)(th % c.heads);
    const int64_t t = th / c.heads;
    const int64_t slot = slots[t];
    const bool write = inside && slot >= 0 && slot < (c.pages << c.shift);
    const int64_t row = c.row(slot >> c.shift, head, (int)(slot & ((1 << c.shift) - 1)));
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
        const uint16_t *src = (kv ? v + t * v_stride : k + t * k_stride) + head * c.D + chunk * 8;
        const uint4 x = load_nt(reinterpret_cast<const uint4 *>(src));
        const uint32_t m = scale_group_max<G / 8>(absmax_bits8(x));
        const float s = quant_scale(h2f((uint16_t)m), 7.0f);
        if (!write)
            continue;
        if (chunk % (G / 8) == 0)
            (kv ? c.vs : c.ks)[row * (c.D / G) + chunk / (G / 8)] = s;
        const uint32_t word = pack_nibbles(quant_chunk8(x, s, 1.0f / s, 7.0f));
        const int g = chunk / 4, b = chunk % 4;
        if (kv == 0) {
            *reinterpret_cast<uint32_t *>(c.k + row * (c.D / 2) + (b * n + g) * 4) = word;
        } else {
            uint8_t *dst = c.v + row * (c.D / 2) + g;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                dst[(4 * b + e) * n] = (uint8_t)(word >> (8 * e));
        }
    }
}

// One lane per 8 elements of a (token, head) row.
__global__ __launch_bounds__(256) void kv4_read_kernel(Kv4Cache c, const int64_t *__restrict__ slots,
                                                       int64_t T, uint16_t *__restrict__ k,
                                                       uint16_t *__restrict__ v)
{
    const int per = c.D / 8, n = c.D / 32;
    const int64_t w = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (w >= T * c.heads * per)
        return;
    const int chunk = (int)(w % per);
    const int64_t th = w / per;
    const int head = (int)(th % c.heads);
    const int64_t slot = slots[th / c.heads];
    const bool there = slot >= 0 && slot < (c.pages << c.shift);
    const int64_t row =
        there ? c.row(slot >> c.shift, head, (int)(slot & ((1 << c.shift) - 1))) : 0;
    const int g = chunk / 4, b = chunk % 4;
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
        uint4 y = make_uint4(0u, 0u, 0u, 0u);
        if (there) {
            const float s = (kv ? c.vs : c.ks)[row * (c.D / c.G) + chunk * 8 / c.G];
            uint32_t word;
            if (kv == 0) {
                word = *reinterpret_cast<const uint32_t *>(c.k + row * (c.D / 2) + (b * n + g) * 4);
            } else {
                const uint8_t *src = c.v + row * (c.D / 2) + g;
                word = 0;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    word |= (uint32_t)src[(4 * b + e) * n] << (8 * e);
            }
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                f[e] = (float)((int32_t)(word << (28 - 4 * e)) >> 28) * s;
            y = make_uint4(pack_h2(f[0], f[1]), pack_h2(f[2], f[3]), pack_h2(f[4], f[5]),
                           pack_h2(f[6], f[7]));
        }
        *reinterpret_cast<uint4 *>((kv ? v : k) + th * c.D + chunk * 8) = y;
    }
}

}  // namespace

void launch_kv4_write(const uint16_t *k, int64_t k_stride, const uint16_t *v, int64_t v_stride,
                      const int64_t *slots, int64_t T, const Kv4Cache &c, hipStream_t st)
{
    const unsigned blocks = (unsigned)((T * c.heads * (c.D / 8) + 255) / 256);
    const auto launch = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3(blocks), dim3(256), 0, st, k, k_stride, v, v_stride, slots,
                           T, c);
    };
    switch (c.G) {
    case 32: launch(kv4_write_kernel<32>); return;
    case 64: launch(kv4_write_kernel<64>); return;
    case 128: launch(kv4_write_kernel<128>); return;
    default: launch(kv4_write_kernel<256>); return;
    }
}

void launch_kv4_read(const Kv4Cache &c, const int64_t *slots, int64_t T, uint16_t *k, uint16_t *v,
                     hipStream_t st)
{
    const unsigned blocks = (unsigned)((T * c.heads * (c.D / 8) + 255) / 256);
    hipLaunchKernelGGL(kv4_read_kernel, dim3(blocks), dim3(256), 0, st, c, slots, T, k, v);
}

}  // namespace w4a8

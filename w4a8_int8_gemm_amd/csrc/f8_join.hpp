// Where the workgroups that share columns of a product in 8-bit floating point
// leave their sums, and how the last of them finishes them.
#pragma once

#include "arrivals.hpp"
#include "f8_device.hpp"
#include "f8.hpp"
#include "kv4.hpp"

namespace w4a8 {

__device__ __forceinline__ float *f8_slot(const F8Args &a, const F8Parts &f, int nb, int split)
{
    return f.sums + ((int64_t)nb * f.splits + split) * a.M * 128;
}

// The 128 columns of block nb from all parts, in order: 32 lanes a token, four
// columns each, four tokens of a thread at a time so that their loads overlap.
__device__ __forceinline__ void f8_join(const F8Args &a, const F8Parts &f, int nb)
{
    constexpr int ROWS = 4;
    const int c4 = 4 * (threadIdx.x & 31);
    const int n = nb * 128 + c4;
    const int there = min(4, a.N - n);                    // columns that are (none or less: nothing was left)
    for (int m0 = threadIdx.x >> 5; m0 < a.M; m0 += 8 * ROWS) {
        float v[ROWS][4] = {};
#pragma unroll 4
        for (int p = 0; p < f.splits; ++p) {
            const float *src = f8_slot(a, f, nb, p) + c4;
            float2 x[ROWS][2];
#pragma unroll
            for (int q = 0; q < ROWS; ++q) {
                const int m = min(m0 + 8 * q, a.M - 1);
                x[q][0] = load_shared(src + m * 128);
                x[q][1] = load_shared(src + m * 128 + 2);
            }
#pragma unroll
            for (int q = 0; q < ROWS; ++q) {
                v[q][0] += x[q][0].x, v[q][1] += x[q][0].y;
                v[q][2] += x[q][1].x, v[q][3] += x[q][1].y;
            }
        }
#pragma unroll
        for (int q = 0; q < ROWS; ++q) {
            const int m = m0 + 8 * q;
            if (m >= a.M)
                break;
            const float *u = v[q];
            if (a.y) {
                uint16_t *p = a.y + (int64_t)m * a.yn + n;
                if (there == 4 && (a.yn & 3) == 0)
                    *reinterpret_cast<uint2 *>(p) = make_uint2(pack_h2(u[0], u[1]), pack_h2(u[2], u[3]));
                else
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (r < there)
                            p[r] = f2h(u[r]);
                continue;
            }
            uint32_t t = 0;
#pragma unroll
            for (int r = 0; r < 4; ++r)
                t = max(t, r < there ? abs_bits(u[r]) : 0u);
            t = group_max_u32<16>(t);
            t = max(t, (uint32_t)__shfl_xor((int)t, 16));
            float s, r;
            f8_block_scale(t, s, r);
            if (c4 == 0)
                a.ys[(int64_t)nb * a.sm + m] = s;
            const uint32_t d = f8_codes4(u[0], u[1], u[2], u[3], s, r);
            uint8_t *p = a.yq + (int64_t)m * a.yn + n;
            if (there == 4 && (a.yn & 3) == 0)
                *reinterpret_cast<uint32_t *>(p) = d;
            else
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (e < there)
                        p[e] = (uint8_t)(d >> (8 * e));
        }
    }
}

}  // namespace w4a8

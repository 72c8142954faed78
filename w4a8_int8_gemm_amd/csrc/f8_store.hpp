// What becomes of a wave's sums in the 8-bit floating point products: the
// activation, fp16 or e4m3, and the stores.
#pragma once

#include "f8.hpp"
#include "f8_device.hpp"
#include "lds_copy.hpp"

namespace w4a8 {

// Exchange between the four lane groups of a wave (lanes 16 g .. 16 g + 15):
// afterwards d[i] of group g is what d[g] of group i was.
__device__ __forceinline__ void transpose_groups(uint32_t (&d)[4])
{
    lane_half_swap(d[0], d[2]);
    lane_half_swap(d[1], d[3]);
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
        const auto r = __builtin_amdgcn_permlane16_swap(d[i], d[i + 1], false, false);
        d[i] = r[0];
        d[i + 1] = r[1];
    }
}

// fp16 of columns n .. n + 15 of row m, eight dwords, clipped to the output.
__device__ __forceinline__ void store_row16(const F8Args &a, int m, int n, const uint32_t (&d)[8])
{
    uint16_t *p = a.y + (int64_t)m * a.N + n;
    if (n + 16 <= a.N && (a.N & 7) == 0) {
        reinterpret_cast<v4u *>(p)[0] = v4u{d[0], d[1], d[2], d[3]};
        reinterpret_cast<v4u *>(p)[1] = v4u{d[4], d[5], d[6], d[7]};
        return;
    }
#pragma unroll
    for (int e = 0; e < 16; ++e)
        if (n + e < a.N)
            p[e] = (uint16_t)(d[e >> 1] >> (16 * (e & 1)));
}

// The sums of MB blocks of 16 tokens and NH blocks of 16 columns of each half:
// lane l holds token m + 16 j + l % 16 and columns 16 i + 4 (l / 16) + r of
// half h in acc[h][i][j][r].
//   m, n      the wave's first token and (first half's) column
//   tile_n    the tile's first column; its second half lies `half` columns on
//   part      which of the waves that share a token's columns this is, of
//             `top`, where they exchange their largest values (e4m3 output:
//             each tile holds 128 columns of a token; all waves of the
//             workgroup call this together); ml = m within the tile
template <bool GATED, int MB, int NH, typename Top>
__device__ __forceinline__ void f8_store_tile(const F8Args &a, float (&acc)[2][NH][MB][4], int m, int n, int tile_n,
                                              int half, int lane, int part, int ml, Top &top)
{
    static_assert(NH == 4, "a lane group stores the columns of one block");
    const int lr = lane & 15, lh = lane >> 4;
    if constexpr (GATED) {
#pragma unroll
        for (int i = 0; i < NH; ++i)
#pragma unroll
            for (int j = 0; j < MB; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    acc[0][i][j][r] = f8_activation(acc[0][i][j][r], a.gelu) * acc[1][i][j][r];
    }
    if (!GATED || a.y) {
#pragma unroll
        for (int h = 0; h < (GATED ? 1 : 2); ++h)
#pragma unroll
            for (int j = 0; j < MB; ++j) {
                uint32_t lo[4], hi[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    lo[i] = pack_h2(acc[h][i][j][0], acc[h][i][j][1]);
                    hi[i] = pack_h2(acc[h][i][j][2], acc[h][i][j][3]);
                }
                transpose_groups(lo);
                transpose_groups(hi);
                const uint32_t d[8] = {lo[0], hi[0], lo[1], hi[1], lo[2], hi[2], lo[3], hi[3]};
                if (m + 16 * j + lr < a.M)
                    store_row16(a, m + 16 * j + lr, n + h * half + 16 * lh, d);
                __builtin_amdgcn_sched_barrier(0);
            }
        return;
    }
    if constexpr (GATED) {
        constexpr int PARTS = sizeof(top) / sizeof(top[0]);
        uint32_t own[MB];
#pragma unroll
        for (int j = 0; j < MB; ++j) {
            uint32_t t = 0;
#pragma unroll
            for (int i = 0; i < NH; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    t = max(t, abs_bits(acc[0][i][j][r]));
            t = max(t, (uint32_t)__shfl_xor((int)t, 16));
            own[j] = max(t, (uint32_t)__shfl_xor((int)t, 32));
        }
        lds_barrier();                                  // `top` of the last tile has been read
#pragma unroll
        for (int j = 0; j < MB; ++j)
            if (lane < 16)
                top[part][ml + 16 * j + lane] = own[j];
        lds_barrier();
#pragma unroll
        for (int j = 0; j < MB; ++j) {
            const int row = m + 16 * j + lr;
            uint32_t t = 0;
#pragma unroll
            for (int p = 0; p < PARTS; ++p)
                t = max(t, top[p][ml + 16 * j + lr]);
            float s, r;
            f8_block_scale(t, s, r);
            uint32_t d[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                d[i] = f8_codes4(acc[0][i][j][0], acc[0][i][j][1], acc[0][i][j][2], acc[0][i][j][3], s, r);
            transpose_groups(d);
            if (row >= a.M)
                continue;
            if (part == 0 && lane < 16)
                a.ys[(int64_t)(tile_n >> 7) * a.M + row] = s;
            const int c = n + 16 * lh;
            uint8_t *p = a.yq + (int64_t)row * a.N + c;
            if (c + 16 <= a.N && (a.N & 15) == 0) {
                *reinterpret_cast<v4u *>(p) = v4u{d[0], d[1], d[2], d[3]};
            } else {
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    if (c + e < a.N)
                        p[e] = (uint8_t)(d[e >> 2] >> (8 * (e & 3)));
            }
        }
    }
}

}  // namespace w4a8

// What becomes of a wave's sums in the 8-bit floating point products: the
// activation, fp16 or e4m3, and the stores.
//
// The sums of MB blocks of 16 tokens and NB blocks of 16 columns: lane l holds
// token 16 j + l % 16 and columns 16 i + 4 (l / 16) + r in acc[i][j][r].
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

// gate := act(gate) * up
template <int NB, int MB>
__device__ __forceinline__ void f8_gate(const F8Args &a, float (&gate)[NB][MB][4], const float (&up)[NB][MB][4])
{
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int j = 0; j < MB; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                gate[i][j][r] = f8_activation(gate[i][j][r], a.gelu) * up[i][j][r];
}

// fp16 outputs of tokens m .., columns n .. (the wave's first).  Four blocks of
// columns are exchanged between the lane groups, so that a lane stores 16
// columns side by side; fewer are stored as they lie, four at a time.
template <int NB, int MB>
__device__ __forceinline__ void f8_store_half(const F8Args &a, const float (&acc)[NB][MB][4], int m, int n, int lane)
{
    const int lr = lane & 15, lh = lane >> 4;
#pragma unroll
    for (int j = 0; j < MB; ++j) {
        const int row = m + 16 * j + lr;
        if constexpr (NB == 4) {
            uint32_t lo[4], hi[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                lo[i] = pack_h2(acc[i][j][0], acc[i][j][1]);
                hi[i] = pack_h2(acc[i][j][2], acc[i][j][3]);
            }
            transpose_groups(lo);
            transpose_groups(hi);
            const int c = n + 16 * lh;
            if (row < a.M) {
                uint16_t *p = a.y + (int64_t)row * a.yn + c;
                if (c + 16 <= a.N && (a.yn & 7) == 0) {
                    reinterpret_cast<v4u *>(p)[0] = v4u{lo[0], hi[0], lo[1], hi[1]};
                    reinterpret_cast<v4u *>(p)[1] = v4u{lo[2], hi[2], lo[3], hi[3]};
                } else {
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        if (c + e < a.N)
                            p[e] = (uint16_t)(((e & 2) ? hi : lo)[e >> 2] >> (16 * (e & 1)));
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        } else if (row < a.M) {
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                const int c = n + 16 * i + 4 * lh;
                uint16_t *p = a.y + (int64_t)row * a.yn + c;
                if (c + 4 <= a.N && (a.yn & 3) == 0)
                    *reinterpret_cast<uint2 *>(p) = make_uint2(pack_h2(acc[i][j][0], acc[i][j][1]),
                                                               pack_h2(acc[i][j][2], acc[i][j][3]));
                else
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (c + r < a.N)
                            p[r] = f2h(acc[i][j][r]);
            }
        }
    }
}

// e4m3 outputs: the workgroup holds the 128 columns from nb * 128 of its
// tokens, this wave those from n; all its waves call this together and exchange
// their largest values in `top` [waves that share a token][tokens of the tile],
// of which this one is `part` and its first token `ml`.
template <int MB, typename Top>
__device__ __forceinline__ void f8_store_f8(const F8Args &a, const float (&acc)[4][MB][4], int m, int n, int nb,
                                            int lane, int part, int ml, Top &top)
{
    constexpr int PARTS = sizeof(top) / sizeof(top[0]);
    const int lr = lane & 15, lh = lane >> 4;
    uint32_t own[MB];
#pragma unroll
    for (int j = 0; j < MB; ++j) {
        uint32_t t = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                t = max(t, abs_bits(acc[i][j][r]));
        t = max(t, (uint32_t)__shfl_xor((int)t, 16));
        own[j] = max(t, (uint32_t)__shfl_xor((int)t, 32));
    }
    lds_barrier();                                      // `top` of the last tile has been read
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
            d[i] = f8_codes4(acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3], s, r);
        transpose_groups(d);
        if (row >= a.M)
            continue;
        if (part == 0 && lane < 16)
            a.ys[(int64_t)nb * a.sm + row] = s;
        const int c = n + 16 * lh;
        uint8_t *p = a.yq + (int64_t)row * a.yn + c;
        if (c + 16 <= a.N && (a.yn & 15) == 0) {
            *reinterpret_cast<v4u *>(p) = v4u{d[0], d[1], d[2], d[3]};
        } else {
#pragma unroll
            for (int e = 0; e < 16; ++e)
                if (c + e < a.N)
                    p[e] = (uint8_t)(d[e >> 2] >> (8 * (e & 3)));
        }
    }
}

}  // namespace w4a8

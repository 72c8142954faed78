// The products in 8-bit floating point for few tokens: the weights streamed
// once (gfx950).
//
// With few tokens a product is bound by reading its weights, so what counts is
// how many of their bytes are on the way at any time:
//
//  * A workgroup owns 16 columns (of the gated pair: the same columns of both
//    weights) and all tokens, and its four waves take the blocks of 128
//    of K in turn.  A wave copies its own blocks straight into its own part of
//    LDS, D - 1 of them ahead of the one it multiplies: no barriers until the
//    waves' sums meet at the end, in fixed order.  A copy takes eight whole
//    128-byte lines of eight rows.
//  * Where a result needs more than one workgroup -- e4m3 output, whose scale
//    is that of 128 columns, or K cut into `splits` ranges because the columns
//    alone do not fill the chip -- the workgroups leave fp32 sums in the
//    workspace, and the last to arrive for 128 columns finishes them, parts in
//    order, so that the result does not depend on who is last.
//
// From HBM: 1 x 4096 x 12288 12.1 us (4.2 TB/s), gated 1 x 12288 x 4096 to fp16
// 23.2 (4.3 TB/s) and in 8 bits, with the workgroups' meeting, 24.2, 32 x 4096 x
// 14336 17.5 (3.4 TB/s), 32 x 10240 x 2560 10.8; that one mostly from the caches
// 7.8, of which 5 to 6 us are those of any launch with its first copies.  From
// 33 tokens on a workgroup's copy of x is larger than its weights: 64 x 4096 x
// 14336 23.9 us (2.5 TB/s).  64 x 64 tiles with K in four read a third of that,
// but their parts have to meet: 22.4 us there, and 13.3 against 8.6 at 64 x 4096
// x 4096, 15.7 against 13.3 at K = 7168.
#include "f8_join.hpp"
#include "lds_copy.hpp"

namespace w4a8 {

namespace {

constexpr int FW = 4;                          // waves

// MB blocks of 16 tokens; HALF: at most 8 tokens, of which only as many rows
// are copied (the other rows of the block repeat them and are dropped).
template <bool GATED, int MB, bool HALF, int D>
__global__ __launch_bounds__(64 * FW) void f8_few_kernel(F8Args a, F8Parts f)
{
    constexpr int SIDES = GATED ? 2 : 1;
    constexpr int XB = HALF ? 1024 : MB * 2048;
    // the scales of a stage: a lane a token and the last two for the weights, or
    // where the tokens need all lanes a copy of their own for the weights'
    constexpr int SC = MB <= 3 ? 1 : 2;
    constexpr int SW = MB <= 3 ? 62 : 64;                   // where the weights' lie
    constexpr int STAGE = XB + SIDES * 2048 + SC * 256;
    constexpr int NI = XB / 1024 + SIDES * 2 + SC;     // copies of a stage
    constexpr int BLOCKS = SIDES * MB;
    constexpr int RED = FW * BLOCKS * 1024;
    constexpr int RING = FW * D * STAGE;
    static_assert((D - 1) * NI < 64, "vmcnt range");
    static_assert(MB <= 4, "a lane a token for its scale");
    __shared__ __attribute__((aligned(1024))) uint8_t lds[RING > RED ? RING : RED];
    __shared__ int last;

    const int M = a.M, N = a.N, K = a.K;
    const int KB = (K + 127) >> 7;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int n0 = (int)blockIdx.x * 16, nb = n0 >> 7;
    const int split = (int)blockIdx.y;
    const bool shared = f.splits > 1 || (GATED && !a.y);    // the result is finished by the last workgroup
    if (shared && threadIdx.x == 0)
        announce(f.counters + (int64_t)nb * kCounterStride, f.tag);

    // this workgroup's blocks of K [k_first, k_first + units), the wave's every fourth
    const int k_first = (int)((int64_t)KB * split / f.splits);
    const int units = (int)((int64_t)KB * (split + 1) / f.splits) - k_first;
    const int nt = wave < units ? (units - 1 - wave) / FW + 1 : 0;

    const int crow = lane >> 3;
    const int chunk0 = 16 * ((lane & 7) ^ crow);
    const v4i rx = make_rsrc(a.x, (uint32_t)(M * K));
    v4i rw[SIDES];
#pragma unroll
    for (int s = 0; s < SIDES; ++s)
        rw[s] = make_rsrc(a.w[s] + (int64_t)n0 * K, (uint32_t)(min(16, N - n0) * K));
    uint8_t *const own = lds + wave * D * STAGE;
    const uint32_t own_at = (uint32_t)__builtin_amdgcn_readfirstlane((int)lds_addr(own));
    // the lane's scale of a stage: tokens first, the weights' in the last lanes
    const float *sc_base;
    int64_t sc_step;
    const float *const sw_base = a.sw[GATED && (lane & 1)] + (int64_t)nb * KB;
    if (SC == 1 && lane >= SW) {
        sc_base = sw_base;
        sc_step = 1;
    } else {
        sc_base = a.sx + min(lane, M - 1);
        sc_step = a.sm;
    }

    const int lr = lane & 15, lh = lane >> 4;
    const int c0 = lh == 0 ? 0 : lh == 1 ? 2 : lh == 2 ? 5 : 7;
    const int sw8 = (lr & 7) ^ (lr >> 3);
    const int fo0 = lr * 128 + 16 * (c0 ^ sw8), fo1 = lr * 128 + 16 * ((c0 ^ 1) ^ sw8);
    const int hr = lr & 7;
    const int ho0 = hr * 128 + 16 * (c0 ^ hr), ho1 = hr * 128 + 16 * ((c0 ^ 1) ^ hr);

    float acc[SIDES][MB][4] = {};

    auto copy = [&](int d, int t) __attribute__((always_inline)) {
        const bool live = t < nt;
        const int u = k_first + (live ? wave + FW * t : 0), k0 = u * 128;
        const uint32_t at = own_at + (uint32_t)(d * STAGE);
        uint32_t vo[2];
#pragma unroll
        for (int par = 0; par < 2; ++par) {
            const int c = chunk0 ^ (16 * par);
            vo[par] = (uint32_t)(crow * K + c) | (!live || k0 + c >= K ? 0x80000000u : 0u);
        }
        const uint32_t kk = (uint32_t)k0;
#pragma unroll
        for (int p = 0; p < XB / 1024; ++p) {
            set_m0(at + p * 1024);
            copy16_buf_to_lds<0>(rx, vo[p & 1] + (uint32_t)(p * 8 * K), kk);
        }
#pragma unroll
        for (int s = 0; s < SIDES; ++s)
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                set_m0(at + XB + (s * 2 + p) * 1024);
                copy16_buf_to_lds<0>(rw[s], vo[p & 1] + (uint32_t)(p * 8 * K), kk);
            }
        copy4_to_lds(sc_base + u * sc_step, at + XB + SIDES * 2048);
        if (SC == 2)
            copy4_to_lds(sw_base + u, at + XB + SIDES * 2048 + 256);
    };
    auto compute = [&](int d) __attribute__((always_inline)) {
        const uint8_t *at = own + d * STAGE;
        auto frag = [&](const uint8_t *p, int o0, int o1) __attribute__((always_inline)) {
            const v4i x = *reinterpret_cast<const v4i *>(p + o0), y = *reinterpret_cast<const v4i *>(p + o1);
            return __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
        };
        const float *sc = reinterpret_cast<const float *>(at + XB + SIDES * 2048);
        v8i xf[MB];
        float sx[MB];
#pragma unroll
        for (int j = 0; j < MB; ++j) {
            xf[j] = HALF ? frag(at, ho0, ho1) : frag(at + j * 2048, fo0, fo1);
            sx[j] = sc[16 * j + lr];
        }
#pragma unroll
        for (int s = 0; s < SIDES; ++s) {
            const float sw = sc[SW + s];
            const v8i wf = frag(at + XB + s * 2048, fo0, fo1);
#pragma unroll
            for (int j = 0; j < MB; ++j) {
                const v4f p = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wf, xf[j], v4f{0, 0, 0, 0},
                                                                               0, 0, 0, 0, 0, 0);
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    acc[s][j][r] = fmaf(p[r], sx[j] * sw, acc[s][j][r]);
            }
        }
    };

#pragma unroll
    for (int d = 0; d < D - 1; ++d)
        copy(d, d);
    int t = 0;
    for (; t + D <= nt; t += D) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
            __builtin_amdgcn_sched_barrier(0);
            copy((d + D - 1) % D, t + d + D - 1);
            wait_vmcnt<(D - 1) * NI>();
            __builtin_amdgcn_sched_barrier(0);
            compute(d);
        }
    }
    __builtin_amdgcn_sched_barrier(0);
    wait_vmcnt<0>();                                  // every copy landed (none may write later)
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int d = 0; d < D - 1; ++d)
        if (t + d < nt)
            compute(d);

    // the waves' sums meet in LDS; wave w finishes the tokens 16 w .. + 15
    lds_barrier();                                    // every wave is done with its stages
    v4f *red = reinterpret_cast<v4f *>(lds);
#pragma unroll
    for (int s = 0; s < SIDES; ++s)
#pragma unroll
        for (int j = 0; j < MB; ++j)
            red[(wave * BLOCKS + s * MB + j) * 64 + lane] = v4f{acc[s][j][0], acc[s][j][1], acc[s][j][2], acc[s][j][3]};
    lds_barrier();
    const int m = 16 * wave + lr, n = n0 + 4 * lh;
    if (wave < MB && m < M && n < N) {
        v4f v[SIDES];
#pragma unroll
        for (int s = 0; s < SIDES; ++s) {
            const int b = s * MB + wave;
            v[s] = red[b * 64 + lane];
#pragma unroll
            for (int y = 1; y < FW; ++y) {
                const v4f u = red[(y * BLOCKS + b) * 64 + lane];
                v[s] = v4f{v[s][0] + u[0], v[s][1] + u[1], v[s][2] + u[2], v[s][3] + u[3]};
            }
        }
        if constexpr (GATED) {
#pragma unroll
            for (int r = 0; r < 4; ++r)
                v[0][r] = f8_activation(v[0][r], a.gelu) * v[1][r];
        }
        if (shared) {
            float *dst = f8_slot(a, f, nb, split) + m * 128 + (n & 127);
            store_shared(dst, v[0][0], v[0][1]);
            store_shared(dst + 2, v[0][2], v[0][3]);
        } else {
            uint16_t *p = a.y + (int64_t)m * a.yn + n;
            if (n + 4 <= N && (a.yn & 3) == 0)
                *reinterpret_cast<uint2 *>(p) = make_uint2(pack_h2(v[0][0], v[0][1]), pack_h2(v[0][2], v[0][3]));
            else
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (n + r < N)
                        p[r] = f2h(v[0][r]);
        }
    }
    if (!shared)
        return;
    __builtin_amdgcn_s_waitcnt(0);                    // this wave's stores are complete
    __syncthreads();
    if (threadIdx.x == 0) {
        const int chunks = (min(128, N - nb * 128) + 15) / 16;
        last = arrive(f.counters + (int64_t)nb * kCounterStride, chunks * f.splits) ? 1 : 0;
    }
    __syncthreads();
    if (last)
        f8_join(a, f, nb);
}

template <bool GATED, int MB, bool HALF>
void launch_few(const F8Args &a, const F8Parts &f, hipStream_t st)
{
    constexpr int STAGE = (HALF ? 1024 : MB * 2048) + (GATED ? 2 : 1) * 2048 + (MB <= 3 ? 256 : 512);
    constexpr int NI = STAGE / 1024 + (MB <= 3 ? 1 : 2);
    // stages as many as the LDS holds of the workgroups that a compute unit gets at once
    constexpr auto depth = [](int per_cu) {
        int d = 156 * 1024 / per_cu / (FW * STAGE);
        d = d < 2 ? 2 : d > 8 ? 8 : d;
        while ((d - 1) * NI >= 64)
            --d;
        return d;
    };
    const dim3 grid((unsigned)((a.N + 15) / 16), (unsigned)f.splits);
    const int64_t groups = (int64_t)grid.x * grid.y;
    if (groups <= a.num_cu)
        hipLaunchKernelGGL((f8_few_kernel<GATED, MB, HALF, depth(1)>), grid, dim3(64 * FW), 0, st, a, f);
    else if (groups <= 2 * a.num_cu)
        hipLaunchKernelGGL((f8_few_kernel<GATED, MB, HALF, depth(2)>), grid, dim3(64 * FW), 0, st, a, f);
    else
        hipLaunchKernelGGL((f8_few_kernel<GATED, MB, HALF, depth(3)>), grid, dim3(64 * FW), 0, st, a, f);
}

template <bool GATED>
void launch_tokens(const F8Args &a, const F8Parts &f, hipStream_t st)
{
    if (a.M <= 8)
        launch_few<GATED, 1, true>(a, f, st);
    else if (a.M <= 16)
        launch_few<GATED, 1, false>(a, f, st);
    else if (a.M <= 32)
        launch_few<GATED, 2, false>(a, f, st);
    else if (a.M <= 48)
        launch_few<GATED, 3, false>(a, f, st);
    else
        launch_few<GATED, 4, false>(a, f, st);
}

}  // namespace

void launch_f8_few(const F8Args &a, bool gated, const F8Parts &f, hipStream_t st)
{
    if (gated)
        launch_tokens<true>(a, f, st);
    else
        launch_tokens<false>(a, f, st);
}

}  // namespace w4a8

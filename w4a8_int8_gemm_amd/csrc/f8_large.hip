// The products in 8-bit floating point for large outputs: 256 x 256 tiles,
// eight waves in two groups that take turns at the matrix unit (gfx950).
#include "f8.hpp"
#include "f8_device.hpp"
#include "f8_store.hpp"
#include "lds_copy.hpp"

namespace w4a8 {

namespace {

constexpr int LBM = 256, LBN = 256;            // tokens and weight rows of a tile
constexpr int LXB = LBM * 128, LWB = LBN * 128;
constexpr int LSB = LXB + LWB;                 // 64 KiB a stage of 128 bytes of K; two stages

// Workgroup barrier without waits or fences of its own: the kernel waits for
// its LDS reads and copies before it.
__device__ __forceinline__ void phase_barrier()
{
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
}

__device__ __forceinline__ void wait_lds()
{
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(15 | (7 << 4) | (0 << 8) | (3 << 14));   // lgkmcnt(0)
    __builtin_amdgcn_sched_barrier(0);
}

template <bool GATED>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2, 2)))
void f8_gemm_large_kernel(F8Args a, int tiles_m, int tiles_n, int group_m)
{
    __shared__ __attribute__((aligned(1024))) uint8_t ring[2 * LSB];
    __shared__ uint32_t top[2][LBM];

    const int M = a.M, N = a.N, K = a.K;
    const int KB = (K + 127) >> 7;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave & 3, group = wave >> 2;       // group: columns 64 group .. + 63 of each half
    constexpr int OUTN = GATED ? 128 : 256;           // output columns of a tile

    const int G = (int)gridDim.x;
    int wl;
    {
        const int bid = (int)blockIdx.x;
        const int xcd = bid & 7, local = bid >> 3;
        const int per = G >> 3, rem = G & 7;
        wl = (xcd < rem) ? xcd * (per + 1) + local : rem * (per + 1) + (xcd - rem) * per + local;
    }
    const int total = tiles_m * tiles_n;
    auto tile_origin = [&](int t, int &m0, int &n0) __attribute__((always_inline)) {
        const int span = group_m * tiles_n;
        const int first_m = (t / span) * group_m;
        const int gm = min(tiles_m - first_m, group_m);
        const int in = t % span;
        m0 = (first_m + in % gm) * LBM;
        n0 = (in / gm) * OUTN;
    };

    // copies: lane l of a 1 KiB block (8 rows) writes row l / 8, place l % 8
    const int chunk0 = 16 * ((lane & 7) ^ (lane >> 3));
    const uint32_t ring_at = (uint32_t)__builtin_amdgcn_readfirstlane((int)lds_addr(ring));
    v4i rx, rw0, rw1;
    auto set_tile = [&](int m0, int n0) __attribute__((always_inline)) {
        rx = make_rsrc(a.x + (int64_t)m0 * K, (uint32_t)(min(LBM, M - m0) * K));
        const int n1 = GATED ? n0 : n0 + 128;
        rw0 = make_rsrc(a.w[0] + (int64_t)n0 * K, (uint32_t)(min(128, N - n0) * K));
        const uint8_t *w1 = GATED ? a.w[1] : a.w[0];
        rw1 = make_rsrc(w1 + (int64_t)min(n1, N) * K, (uint32_t)(max(0, min(128, N - n1)) * K));
    };
    // group 0 copies: its wave wm takes blocks 8 wm .. + 7 of X and of W (4 of each half)
    auto issue_stage = [&](int s) __attribute__((always_inline)) {
        const uint32_t k0 = (uint32_t)(s * 128);
        const uint32_t base = ring_at + (uint32_t)((s & 1) * LSB);
        int ch = chunk0;
        asm volatile("" : "+v"(ch));       // the offsets are formed here each time, not kept in registers
        uint32_t vo[2];
#pragma unroll
        for (int par = 0; par < 2; ++par) {
            const int c = ch ^ (16 * par);
            // chunks past the row's end (the last stage of a K that 128 does not divide) read zeros
            vo[par] = (uint32_t)((lane >> 3) * K + c) | ((int)k0 + c >= K ? 0x80000000u : 0u);
        }
#pragma unroll
        for (int p = 0; p < 8; ++p) {
            const int blk = wm * 8 + p;
            set_m0(base + blk * 1024);
            copy16_buf_to_lds<0>(rx, vo[p & 1] + (uint32_t)(blk * 8 * K), k0);
        }
#pragma unroll
        for (int p = 0; p < 8; ++p) {
            const int blk = wm * 4 + (p & 3);
            set_m0(base + LXB + (p >> 2) * 16384 + blk * 1024);
            copy16_buf_to_lds<0>(p < 4 ? rw0 : rw1, vo[p & 1] + (uint32_t)(blk * 8 * K), k0);
        }
    };

    // fragments: lane l reads row l % 16; of the eight 16-byte chunks of a
    // stage lane group h takes 0 1, 2 3, 5 4, 7 6
    const int lr = lane & 15, lh = lane >> 4;
    const int c0 = lh == 0 ? 0 : lh == 1 ? 2 : lh == 2 ? 5 : 7;
    const int sw8 = (lr & 7) ^ (lr >> 3);
    const int fo0 = lr * 128 + 16 * (c0 ^ sw8), fo1 = lr * 128 + 16 * ((c0 ^ 1) ^ sw8);
    auto read_frag = [&](const uint8_t *rows) __attribute__((always_inline)) {
        const v4i p = *reinterpret_cast<const v4i *>(rows + fo0), q = *reinterpret_cast<const v4i *>(rows + fo1);
        return __builtin_shufflevector(p, q, 0, 1, 2, 3, 4, 5, 6, 7);
    };

    float acc[2][4][4][4];
    v8i xf[4], wf[4];
    v4f pr[4];
    float sc[2][4];

    // sixteen products of one half, each folded three products later
    auto compute = [&](auto HALF) __attribute__((always_inline)) {
        constexpr int h = decltype(HALF)::value;
#pragma unroll
        for (int t = 0; t < 16 + 3; ++t) {
            if (t < 16)
                pr[t & 3] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wf[t >> 2], xf[t & 3], v4f{0, 0, 0, 0},
                                                                             0, 0, 0, 0, 0, 0);
            __builtin_amdgcn_sched_barrier(0);
            if (t >= 3) {
                const int u = t - 3;
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    acc[h][u >> 2][u & 3][r] = fmaf(pr[u & 3][r], sc[h][u & 3], acc[h][u >> 2][u & 3][r]);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    };

    int tile = wl;
    int m0, n0;
    tile_origin(tile, m0, n0);
    set_tile(m0, n0);
    if (group == 0) {
        issue_stage(0);
    }
    while (true) {
        const int nb = n0 >> 7, nb1 = GATED ? nb : min(nb + 1, ((N + 127) >> 7) - 1);
        const float *swp0 = a.sw[0] + (int64_t)nb * KB, *swp1 = a.sw[GATED] + (int64_t)nb1 * KB;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        acc[h][i][j][r] = 0.0f;
        float sx[4], sw[2];
        auto load_scales = [&](int s) __attribute__((always_inline)) {
            const char *row = reinterpret_cast<const char *>(a.sx + (int64_t)s * M);
            uint32_t at = lr;
            asm volatile("" : "+v"(at));       // as above
#pragma unroll
            for (int j = 0; j < 4; ++j)
                sx[j] = *reinterpret_cast<const float *>(row + 4 * min(at + (uint32_t)(m0 + wm * 64 + 16 * j), (uint32_t)M - 1));
            at = 0;
            asm volatile("" : "+v"(at));       // the weights' scales by vector loads too: scalar ones and LDS reads
            sw[0] = *reinterpret_cast<const float *>(reinterpret_cast<const char *>(swp0 + s) + at);   // share a counter
            sw[1] = *reinterpret_cast<const float *>(reinterpret_cast<const char *>(swp1 + s) + at);
        };
        load_scales(0);
        wait_vmcnt<0>();
        phase_barrier();
        if (group == 1)
            phase_barrier();
#pragma clang loop unroll(disable)
        for (int s = 0; s < KB; ++s) {
            const uint8_t *buf = ring + (s & 1) * LSB;
            const uint8_t *xb = buf + wm * 64 * 128, *wb = buf + LXB + group * 64 * 128;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                xf[i] = read_frag(xb + i * 2048);
                wf[i] = read_frag(wb + i * 2048);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    sc[h][j] = sx[j] * sw[h];
            __builtin_amdgcn_sched_barrier(0);
            load_scales(min(s + 1, KB - 1));
            if (group == 0 && s + 1 < KB)
                issue_stage(s + 1);
            wait_lds();
            phase_barrier();
            compute(std::integral_constant<int, 0>());
            phase_barrier();
#pragma unroll
            for (int i = 0; i < 4; ++i)
                wf[i] = read_frag(wb + 16384 + i * 2048);
            wait_lds();
            phase_barrier();
            compute(std::integral_constant<int, 1>());
            __builtin_amdgcn_sched_barrier(0);
            wait_vmcnt<0>();
            phase_barrier();
        }
        if (group == 0)
            phase_barrier();
        // both groups are past their last reads: the next tile's stages may come
        const int om = m0, on = n0;
        tile += G;
        const bool more = tile < total;
        if (more) {
            tile_origin(tile, m0, n0);
            set_tile(m0, n0);
            if (group == 0) {
                issue_stage(0);
            }
        }
        f8_store_tile<GATED, 4, 4>(a, acc, om + wm * 64, on + group * 64, on, 128, lane, group, wm * 64, top);
        if (!more)
            break;
    }
    wait_vmcnt<0>();
}

}  // namespace

template <bool GATED>
static void launch_large(const F8Args &a, hipStream_t st)
{
    const int tiles_m = (a.M + LBM - 1) / LBM, tiles_n = (a.N + (GATED ? 127 : 255)) / (GATED ? 128 : 256);
    const int64_t tiles = (int64_t)tiles_m * tiles_n;
    const int grid = (int)(tiles < a.num_cu ? tiles : a.num_cu);
    hipLaunchKernelGGL(f8_gemm_large_kernel<GATED>, dim3(grid), dim3(512), 0, st, a, tiles_m, tiles_n, 4);
}

void launch_f8_large(const F8Args &a, bool gated, hipStream_t st)
{
    if (gated)
        launch_large<true>(a, st);
    else
        launch_large<false>(a, st);
}

}  // namespace w4a8

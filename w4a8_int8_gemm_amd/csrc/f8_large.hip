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

// At most N of the wave's copies may still be on their way.
template <int N> __device__ __forceinline__ void wait_copies()
{
    __builtin_amdgcn_sched_barrier(0);
    wait_vmcnt<N>();
    __builtin_amdgcn_sched_barrier(0);
}

template <bool GATED>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2, 2)))
void f8_gemm_large_kernel(F8Args a, int tiles_m, int tiles_n, int group_m)
{
    __shared__ __attribute__((aligned(1024))) uint8_t ring[2 * LSB];
    __shared__ __attribute__((aligned(256))) float scales[2][2][LBM];   // [stage parity][of x, of w][4 waves x 64]
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

    // ---- copies.  The stages of all of the workgroup's tiles are one stream;
    // the cursor is the stage whose x and first half of w come next, the
    // second half follows one stage later (its own resource and k).  Lane l of
    // a 1 KiB block (8 rows) writes row l / 8, place l % 8.
    const int chunk0 = 16 * ((lane & 7) ^ (lane >> 3));
    const uint32_t ring_at = (uint32_t)__builtin_amdgcn_readfirstlane((int)lds_addr(ring));
    const uint32_t scales_at = (uint32_t)__builtin_amdgcn_readfirstlane((int)lds_addr(scales));
    v4i rx, rw0, rw1, rw1_now;
    const float *scp;
    int cur_tile = wl, cur_s = 0, cur_m0, w1_s = 0;
    uint32_t cur_buf = 0;
    auto set_tile = [&]() __attribute__((always_inline)) {
        int m0, n0;
        tile_origin(cur_tile, m0, n0);
        cur_m0 = m0;
        rx = make_rsrc(a.x + (int64_t)m0 * K, (uint32_t)(min(LBM, M - m0) * K));
        const int n1 = GATED ? n0 : n0 + 128;
        rw0 = make_rsrc(a.w[0] + (int64_t)n0 * K, (uint32_t)(min(128, N - n0) * K));
        rw1 = make_rsrc(a.w[GATED] + (int64_t)min(n1, N) * K, (uint32_t)(max(0, min(128, N - n1)) * K));
        const int nb = n0 >> 7, nb1 = GATED ? nb : min(nb + 1, ((N + 127) >> 7) - 1);
        if (group == 0)
            scp = a.sx + min(m0 + wave * 64, M - 1);
        else
            scp = a.sw[GATED && (wave & 1)] + (int64_t)((wave & 1) ? nb1 : nb) * KB;
    };
    auto advance = [&]() __attribute__((always_inline)) {
        rw1_now = rw1;
        w1_s = cur_s;
        cur_buf ^= 1;
        if (cur_s + 1 < KB) {
            ++cur_s;
        } else if (cur_tile + G < total) {            // past the end: the last stage again
            cur_s = 0;
            cur_tile += G;
            set_tile();
        }
    };
    // A lane's offset in a block of even (par 0) or odd number; chunks past the
    // row's end (the last stage of a K that 128 does not divide) read zeros.
    // Formed each time, not kept in registers.
    auto lane_offset = [&](int par, int k0) __attribute__((always_inline)) {
        int ch = chunk0;
        asm volatile("" : "+v"(ch));
        const int c = ch ^ (16 * par);
        return (uint32_t)((lane >> 3) * K + c) | (k0 + c >= K ? 0x80000000u : 0u);
    };
    auto copy_x = [&](int p) __attribute__((always_inline)) {         // p = 0 .. 3
        const int blk = wave * 4 + p, k0 = cur_s * 128;
        set_m0(ring_at + cur_buf * LSB + blk * 1024);
        copy16_buf_to_lds<0>(rx, lane_offset(p & 1, k0) + (uint32_t)(blk * 8 * K), (uint32_t)k0);
    };
    auto copy_w0 = [&](int p) __attribute__((always_inline)) {        // p = 0, 1
        const int blk = wave * 2 + p, k0 = cur_s * 128;
        set_m0(ring_at + cur_buf * LSB + LXB + blk * 1024);
        copy16_buf_to_lds<0>(rw0, lane_offset(p, k0) + (uint32_t)(blk * 8 * K), (uint32_t)k0);
    };
    auto copy_w1 = [&](int p) __attribute__((always_inline)) {        // of the stage before the cursor's
        const int blk = wave * 2 + p, k0 = w1_s * 128;
        set_m0(ring_at + (cur_buf ^ 1) * LSB + LXB + 16384 + blk * 1024);
        copy16_buf_to_lds<0>(rw1_now, lane_offset(p, k0) + (uint32_t)(blk * 8 * K), (uint32_t)k0);
    };
    // waves 0-3: x's scales of 64 tokens; wave 4 (and 6): the first half's of
    // w, wave 5 (and 7): the second's, in every lane
    const int64_t sc_step = group == 0 ? a.sm : 1;
    const uint32_t sc_mask = group == 0 ? 63 : 0;
    auto copy_scales = [&]() __attribute__((always_inline)) {
        uint32_t l = (uint32_t)lane & sc_mask;
        asm volatile("" : "+v"(l));
        l = min(l, (uint32_t)max(0, M - 1 - cur_m0 - wm * 64));
        copy4_to_lds(scp + cur_s * sc_step + l, scales_at + cur_buf * 2048 + wave * 256);
    };

    // ---- fragments: lane l reads row l % 16; of the eight 16-byte chunks of a
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

    // sixteen products of one half, each folded three products later; `copy`
    // runs between them
    auto compute = [&](auto HALF, auto copy) __attribute__((always_inline)) {
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
            if (t < 16)
                copy(t);
            __builtin_amdgcn_sched_barrier(0);
        }
        // the sums are formed here, not where the compiler next needs them
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float *v = acc[h][i][j];
                asm volatile("" : "+v"(v[0]), "+v"(v[1]), "+v"(v[2]), "+v"(v[3]));
            }
    };

    set_tile();
#pragma unroll
    for (int p = 0; p < 4; ++p)
        copy_x(p);
    copy_w0(0);
    copy_w0(1);
    copy_scales();
    advance();
    copy_w1(0);
    copy_w1(1);
#pragma unroll
    for (int p = 0; p < 4; ++p)
        copy_x(p);
    copy_w0(0);
    copy_w0(1);
    copy_scales();
    wait_vmcnt<9>();                                  // the first stage's x, w0 and scales
    phase_barrier();
    int b = 0;
    for (int tile = wl; tile < total; tile += G) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        acc[h][i][j][r] = 0.0f;
        if (group == 1)
            phase_barrier();
#pragma clang loop unroll(disable)
        for (int s = 0; s < KB; ++s) {
            const uint8_t *buf = ring + b * LSB;
            const uint8_t *xb = buf + wm * 64 * 128, *wb = buf + LXB + group * 64 * 128;
            float sx[4], sw[2];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                xf[i] = read_frag(xb + i * 2048);
                wf[i] = read_frag(wb + i * 2048);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
                sx[j] = scales[b][0][wm * 64 + 16 * j + lr];
            sw[0] = scales[b][1][0];
            sw[1] = scales[b][1][64];
            __builtin_amdgcn_sched_barrier(0);
            advance();
            copy_w1(0);
            wait_lds();
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    sc[h][j] = sx[j] * sw[h];
            wait_copies<8>();                         // this stage's second half of w
            phase_barrier();
            compute(std::integral_constant<int, 0>(), [&](int t) __attribute__((always_inline)) {
                if (t == 4)
                    copy_w1(1);
            });
            phase_barrier();
#pragma unroll
            for (int i = 0; i < 4; ++i)
                wf[i] = read_frag(wb + 16384 + i * 2048);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int p = 0; p < 4; ++p)
                copy_x(p);
            wait_lds();
            wait_copies<6>();                         // the next stage's x, first half of w and scales
            phase_barrier();
            compute(std::integral_constant<int, 1>(), [&](int t) __attribute__((always_inline)) {
                if (t == 2 || t == 6)
                    copy_w0(t >> 2);
                if (t == 10)
                    copy_scales();
            });
            phase_barrier();
            b ^= 1;
        }
        if (group == 0)
            phase_barrier();
        int m0, n0;
        tile_origin(tile, m0, n0);
        const int mw = m0 + wm * 64, nw = n0 + group * 64;
        if constexpr (GATED) {
            f8_gate(a, acc[0], acc[1]);
            if (a.y)
                f8_store_half(a, acc[0], mw, nw, lane);
            else
                f8_store_f8(a, acc[0], mw, nw, n0 >> 7, lane, group, wm * 64, top);
        } else {
            f8_store_half(a, acc[0], mw, nw, lane);
            f8_store_half(a, acc[1], mw, nw + 128, lane);
        }
    }
    wait_vmcnt<0>();                                  // no copy may still be writing LDS at the end
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

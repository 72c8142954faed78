// The products in 8-bit floating point for tens to hundreds of tokens: small
// tiles, their stages in a deep ring (gfx950).
//
// Where the output has too few tiles for the large ones, a workgroup's time is
// that of bringing its operands into LDS and of the latency of each stage.  So:
// tiles small enough to fill the chip, a ring of D stages of 128 bytes of K that
// the four waves fill together, up to D - 1 of them on the way, one barrier a
// stage, the next stage's fragments read while one is multiplied.  With 64
// columns and e4m3 output two workgroups share a scale; they meet as those of
// f8_few.hip do.  Where the tiles are few, workgroups take parts of K.
//
// 517 x 4096 x 4096 17.4 us (1000 TFLOP/s; 21 with its quantizer), 300 x 5120 x
// 2560 11.1 us and the gated pair 301 x 5121 x 2560 17.8 (890 TFLOP/s): 5.5 us of
// each are a launch's start and end, the rest 0.28 to 0.6 us a stage, in which
// a workgroup brings 53 to 77 KB/us.  Two on one compute unit bring 125
// together, so it is not the unit's rate that bounds these, which have one
// each, but what four waves with a barrier a stage keep on the way; eight
// waves a workgroup have not been tried.
#include "f8_join.hpp"
#include "f8_store.hpp"

namespace w4a8 {

namespace {

// WM x WN waves of MB blocks of 16 tokens and, of each side, NB blocks of 16
// columns.
template <bool GATED, int WM, int WN, int MB, int NB, int D>
__global__ __launch_bounds__(256) void f8_tile_kernel(F8Args a, F8Parts f, int tiles_m)
{
    constexpr int SIDES = GATED ? 2 : 1;
    constexpr int BM = 16 * WM * MB, RS = 16 * WN * NB;     // tokens, columns
    constexpr int XC = BM / 8, WC = RS / 8;                 // copies of 1 KiB
    constexpr int DATA = (XC + SIDES * WC) * 1024;
    constexpr int STAGE = DATA + 1024;                      // and 4 x 64 scales
    constexpr int NI = (XC + SIDES * WC) / 4 + 1;           // copies of a wave
    static_assert(WM * WN == 4 && XC % 4 == 0 && WC % 4 == 0, "the waves copy equal shares");
    static_assert(BM <= 128 && RS <= 128 && 128 % RS == 0, "two copies of scales, one block of weights");
    static_assert(D >= 2 && (D - 1) * NI < 64, "vmcnt range");
    __shared__ __attribute__((aligned(1024))) uint8_t ring[D * STAGE];
    __shared__ uint32_t top[WN][BM];
    __shared__ int last;

    const int M = a.M, N = a.N, K = a.K;
    const int KB = (K + 127) >> 7;
    // this workgroup's range of K
    const int split = (int)blockIdx.y;
    const int k_first = (int)((int64_t)KB * split / f.splits), k_end = (int)((int64_t)KB * (split + 1) / f.splits);
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int wm = wave % WM, wn = wave / WM;

    // the workgroups of one XCD (blockIdx % 8) take neighbouring tiles: the
    // token tiles of the same columns, then the next columns
    int id;
    {
        const int G = (int)gridDim.x, bid = (int)blockIdx.x;
        const int xcd = bid & 7, local = bid >> 3, per = G >> 3, rem = G & 7;
        id = (xcd < rem) ? xcd * (per + 1) + local : rem * (per + 1) + (xcd - rem) * per + local;
    }
    const int m0 = id % tiles_m * BM;
    const int n0 = id / tiles_m * RS, nb = n0 >> 7;
    const bool shared = GATED && RS < 128 && !a.y;         // one tile of tokens: launch_f8()
    if (shared && threadIdx.x == 0)
        announce(f.counters + (int64_t)nb * kCounterStride, f.tag);
    if (f.splits > 1 && threadIdx.x == 0)
        announce(f.counters + (int64_t)id * kCounterStride, f.tag);

    const int crow = lane >> 3;
    const int chunk0 = 16 * ((lane & 7) ^ crow);
    const v4i rx = make_rsrc(a.x + (int64_t)m0 * K, (uint32_t)(min(BM, M - m0) * K));
    v4i rw[SIDES];
#pragma unroll
    for (int s = 0; s < SIDES; ++s)
        rw[s] = make_rsrc(a.w[s] + (int64_t)n0 * K, (uint32_t)(min(RS, N - n0) * K));
    const uint32_t ring_at = (uint32_t)__builtin_amdgcn_readfirstlane((int)lds_addr(ring));
    // waves 0 and 1: x's scales of 64 tokens each; waves 2 and 3: w's of a side, in every lane
    const float *const sc_base = wave < 2 ? a.sx + min(m0 + wave * 64 + lane, M - 1)
                                          : a.sw[GATED && wave == 3] + (int64_t)nb * KB;
    const int64_t sc_step = wave < 2 ? a.sm : 1;

    // copy p of the wave's of a stage into its slot: XC / 4 blocks of 8 rows of
    // x, WC / 4 of each side of w, the scales; past the last stage nothing is fetched
    struct Stage {
        uint32_t at, x[2], w[2], k0;
        int u;
    };
    const int xblk = wave * (XC / 4), wblk = wave * (WC / 4);
    auto stage_of = [&](int slot, int t) __attribute__((always_inline)) {
        const bool live = t < k_end;
        Stage g;
        g.u = live ? t : k_first;
        g.k0 = (uint32_t)(g.u * 128);
        g.at = ring_at + (uint32_t)(slot * STAGE);
        const int end = live ? K - (int)g.k0 : 0;          // bytes of a row from this stage on
#pragma unroll
        for (int par = 0; par < 2; ++par) {
            const int cx = chunk0 ^ (16 * ((par + xblk) & 1)), cw = chunk0 ^ (16 * ((par + wblk) & 1));
            g.x[par] = (uint32_t)((crow + 8 * xblk) * K + cx) | (cx >= end ? 0x80000000u : 0u);
            g.w[par] = (uint32_t)((crow + 8 * wblk) * K + cw) | (cw >= end ? 0x80000000u : 0u);
        }
        return g;
    };
    auto copy = [&](const Stage &g, int p) __attribute__((always_inline)) {
        if (p == NI - 1) {
            copy4_to_lds(sc_base + g.u * sc_step, g.at + DATA + wave * 256);
        } else if (p < XC / 4) {
            set_m0(g.at + (xblk + p) * 1024);
            copy16_buf_to_lds<0>(rx, g.x[p & 1] + (uint32_t)(p * 8 * K), g.k0);
        } else {
            const int side = (p - XC / 4) / (WC / 4), q = (p - XC / 4) % (WC / 4);
            set_m0(g.at + (XC + side * WC + wblk + q) * 1024);
            copy16_buf_to_lds<0>(rw[side], g.w[q & 1] + (uint32_t)(q * 8 * K), g.k0);
        }
    };

    const int lr = lane & 15, lh = lane >> 4;
    const int c0 = lh == 0 ? 0 : lh == 1 ? 2 : lh == 2 ? 5 : 7;
    const int sw8 = (lr & 7) ^ (lr >> 3);
    const int fo0 = lr * 128 + 16 * (c0 ^ sw8), fo1 = lr * 128 + 16 * ((c0 ^ 1) ^ sw8);
    auto frag = [&](const uint8_t *p) __attribute__((always_inline)) {
        const v4i x = *reinterpret_cast<const v4i *>(p + fo0), y = *reinterpret_cast<const v4i *>(p + fo1);
        return __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
    };

    float acc[SIDES][NB][MB][4];
#pragma unroll
    for (int s = 0; s < SIDES; ++s)
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
            for (int j = 0; j < MB; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    acc[s][i][j][r] = 0.0f;

    // Fragments and scales of a stage, read while the one before is multiplied.
    struct Frags {
        v8i x[MB], w[SIDES][NB];
        float sx[MB], sw[SIDES];
    };
    constexpr int READS = MB + SIDES * NB;
    auto read = [&](Frags &F, int slot, int q) __attribute__((always_inline)) {
        const uint8_t *at = ring + slot * STAGE;
        const float *sc = reinterpret_cast<const float *>(at + DATA);
        if (q < MB) {
            F.x[q] = frag(at + (wm * MB + q) * 2048);
            F.sx[q] = sc[(wm * MB + q) * 16 + lr];
        } else {
            const int s = (q - MB) / NB, i = (q - MB) % NB;
            F.w[s][i] = frag(at + XC * 1024 + s * WC * 1024 + (wn * NB + i) * 2048);
            if (i == 0)
                F.sw[s] = sc[128 + 64 * s];
        }
    };
    constexpr int COUNT = SIDES * NB * MB;                 // products of a wave and stage
    constexpr int LAG = COUNT >= 8 ? 3 : 1;                // folded so many products later
    auto multiply = [&](const Frags &F, const Stage &g, Frags &then, int slot) __attribute__((always_inline)) {
        v4f pr[LAG + 1];
        float sm[SIDES][MB];
#pragma unroll
        for (int s = 0; s < SIDES; ++s)
#pragma unroll
            for (int j = 0; j < MB; ++j)
                sm[s][j] = F.sx[j] * F.sw[s];
#pragma unroll
        for (int t = 0; t < COUNT + LAG; ++t) {
            if (t < COUNT)
                pr[t % (LAG + 1)] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                    F.w[t / (NB * MB)][t / MB % NB], F.x[t % MB], v4f{0, 0, 0, 0}, 0, 0, 0, 0, 0, 0);
            __builtin_amdgcn_sched_barrier(0);
            if (t >= LAG) {
                const int u = t - LAG, s = u / (NB * MB), i = u / MB % NB, j = u % MB;
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    acc[s][i][j][r] = fmaf(pr[u % (LAG + 1)][r], sm[s][j], acc[s][i][j][r]);
            }
            // the copies, spread over the products, and the reads, over the first half of them
#pragma unroll
            for (int p = 0; p < (NI > READS ? NI : READS); ++p) {
                if (t < COUNT && p < NI && p * COUNT / NI == t)
                    copy(g, p);
                if (t < COUNT && p < READS && p * ((COUNT + 1) / 2) / READS == t)
                    read(then, slot, p);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    // Stage t's place is free again once everyone has read it, which the
    // barrier of iteration t says (the reads end before it: lds_barrier waits).
    auto step = [&](Frags &now, Frags &then, int &slot, int t) __attribute__((always_inline)) {
        __builtin_amdgcn_sched_barrier(0);
        wait_vmcnt<(D - 2) * NI>();                        // the wave's share of stage t + 1 has landed
        lds_barrier();
        const Stage g = stage_of(slot, t + D);
        slot = slot + 1 == D ? 0 : slot + 1;
        multiply(now, g, then, slot);
    };

#pragma unroll
    for (int d = 0; d < D; ++d) {
        const Stage g = stage_of(d, k_first + d);
#pragma unroll
        for (int p = 0; p < NI; ++p)
            copy(g, p);
    }
    int slot = 0;
    Frags f0, f1;
    wait_vmcnt<(D - 1) * NI>();
    lds_barrier();
#pragma unroll
    for (int q = 0; q < READS; ++q)
        read(f0, 0, q);
    for (int t = k_first; t < k_end; t += 2) {
        step(f0, f1, slot, t);
        if (t + 1 < k_end)
            step(f1, f0, slot, t + 1);
    }
    wait_vmcnt<0>();                                       // no copy may still be writing LDS at the end

    // K in parts: each leaves its sums as its threads hold them, the last to
    // arrive adds them up in their order and goes on as the only one
    if (f.splits > 1) {
        constexpr int SUMS = SIDES * NB * MB * 4 * 256;
        const int64_t tiles = gridDim.x;
        float *const at = f.sums + (int64_t)id * SUMS + 2 * threadIdx.x;
#pragma unroll
        for (int s = 0; s < SIDES; ++s)
#pragma unroll
            for (int i = 0; i < NB; ++i)
#pragma unroll
                for (int j = 0; j < MB; ++j)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        store_shared(at + split * tiles * SUMS + (((s * NB + i) * MB + j) * 2 + h) * 512,
                                     acc[s][i][j][2 * h], acc[s][i][j][2 * h + 1]);
        __builtin_amdgcn_s_waitcnt(0);                     // this wave's stores are complete
        __syncthreads();
        if (threadIdx.x == 0)
            last = arrive(f.counters + (int64_t)id * kCounterStride, f.splits) ? 1 : 0;
        __syncthreads();
        if (!last)
            return;
#pragma unroll
        for (int s = 0; s < SIDES; ++s)
#pragma unroll
            for (int i = 0; i < NB; ++i)
#pragma unroll
                for (int j = 0; j < MB; ++j)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        acc[s][i][j][r] = 0.0f;
        for (int p = 0; p < f.splits; ++p) {
            const float *from = at + p * tiles * SUMS;
#pragma unroll
            for (int s = 0; s < SIDES; ++s)
#pragma unroll
                for (int i = 0; i < NB; ++i) {
                    float2 v[MB][2];
#pragma unroll
                    for (int j = 0; j < MB; ++j)
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            v[j][h] = load_shared(from + (((s * NB + i) * MB + j) * 2 + h) * 512);
#pragma unroll
                    for (int j = 0; j < MB; ++j)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            acc[s][i][j][2 * h] += v[j][h].x;
                            acc[s][i][j][2 * h + 1] += v[j][h].y;
                        }
                }
        }
    }

    const int mw = m0 + wm * MB * 16, nw = n0 + wn * NB * 16;
    if constexpr (GATED)
        f8_gate(a, acc[0], acc[1]);
    if (!shared) {
        if constexpr (GATED && RS == 128 && NB == 4) {
            if (!a.y) {
                f8_store_f8(a, acc[0], mw, nw, nb, lane, wn, wm * MB * 16, top);
                return;
            }
        }
        f8_store_half(a, acc[0], mw, nw, lane);
        return;
    }
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int j = 0; j < MB; ++j) {
            const int m = mw + 16 * j + lr, n = nw + 16 * i + 4 * lh;
            if (m < M && n < N) {
                float *dst = f8_slot(a, f, nb, 0) + m * 128 + (n & 127);
                store_shared(dst, acc[0][i][j][0], acc[0][i][j][1]);
                store_shared(dst + 2, acc[0][i][j][2], acc[0][i][j][3]);
            }
        }
    __builtin_amdgcn_s_waitcnt(0);                         // this wave's stores are complete
    __syncthreads();
    if (threadIdx.x == 0)
        last = arrive(f.counters + (int64_t)nb * kCounterStride, (min(128, N - nb * 128) + RS - 1) / RS) ? 1 : 0;
    __syncthreads();
    if (last)
        f8_join(a, f, nb);
}

template <bool GATED, int WM, int WN, int MB, int NB>
void launch_tile(const F8Args &a, const F8Parts &f, hipStream_t st)
{
    constexpr int BM = 16 * WM * MB, RS = 16 * WN * NB;
    constexpr int STAGE = (BM + (GATED ? 2 : 1) * RS) * 128 + 1024;
    constexpr int NI = (BM + (GATED ? 2 : 1) * RS) / 32 + 1;
    const int tiles_m = (a.M + BM - 1) / BM;
    const dim3 grid((unsigned)(tiles_m * ((a.N + RS - 1) / RS)), (unsigned)f.splits);
    // stages as many as half of a compute unit's LDS holds, or where the grid
    // has one workgroup for each (or half holds fewer than two), all of it
    constexpr auto depth = [](int bytes) {
        int d = bytes / STAGE < 8 ? bytes / STAGE : 8;
        while ((d - 1) * NI >= 64)
            --d;
        return d;
    };
    constexpr int ALL = depth(157 * 1024), PART = depth(78 * 1024) < 2 ? ALL : depth(78 * 1024);
    if ((int64_t)grid.x * grid.y <= a.num_cu)
        hipLaunchKernelGGL((f8_tile_kernel<GATED, WM, WN, MB, NB, ALL>), grid, dim3(256), 0, st, a, f, tiles_m);
    else
        hipLaunchKernelGGL((f8_tile_kernel<GATED, WM, WN, MB, NB, PART>), grid, dim3(256), 0, st, a, f, tiles_m);
}

template <bool GATED>
void launch_shapes(const F8Args &a, int shape, const F8Parts &f, hipStream_t st)
{
    switch (shape) {                                       // kF8Tiles
    case 0: launch_tile<GATED, 1, 4, 4, 1>(a, f, st); return;
    case 1: launch_tile<GATED, 2, 2, 2, 4>(a, f, st); return;
    case 2: launch_tile<GATED, 2, 2, 3, 4>(a, f, st); return;
    case 3: launch_tile<GATED, 2, 2, 4, 2>(a, f, st); return;
    default: launch_tile<GATED, 2, 2, 4, 4>(a, f, st); return;
    }
}

}  // namespace

void launch_f8_tile(const F8Args &a, bool gated, int shape, const F8Parts &f, hipStream_t st)
{
    if (gated)
        launch_shapes<true>(a, shape, f, st);
    else
        launch_shapes<false>(a, shape, f, st);
}

}  // namespace w4a8

// The products in 8-bit floating point for large outputs (gfx950): y = sum over
// blocks b of 128 of K of (sx[b, m] sw[n / 128, b]) (x_b . w_b), 256 x 256 tiles
// of it by eight waves, of the gated pair 256 x 128 of both.
//
// Bound by the matrix unit, which may not wait: a 16 x 16 x 128 product is 32
// cycles of it, and its sums' scales change with each, so that each is folded
// into fp32 sums by four multiply-adds.  A loop of only these two, operands in
// registers, takes 40 cycles a product (3810 TFLOP/s over the chip, 4770 without
// the folds); here it is 46, with copies, reads and barriers, and the clock
// falls to 1.84 GHz under the load.  What that takes:
//  * A wave owns 64 tokens x 64 columns of each half of the tile: 32 products a
//    stage from 12 fragments, all 128 sums and the fragments in registers.  A
//    wave with half the columns would read half as much again from LDS.
//  * A product is issued, then the fold of the third before it, whose result
//    is there; fragments are replaced as soon as their last product is issued
//    and the copies spread between, two stages of 64 KiB, so that no stretch
//    waits for LDS.  Two barriers a stage: behind the wait for a stage's second
//    half of w, and for the next stage's x and first half.  They keep the two
//    waves of a SIMD within a half stage of each other and no closer; fixed
//    turns between them cost more than they gave (8192^3 456 us, with the
//    fragments read one stage ahead 466; without any 429).
//  * Resources, offsets and places are held, not recomputed: 470 us otherwise.
//  * The stages of all of a workgroup's tiles are one stream, so the next
//    tile's first stages are on their way while the last one's sums are stored.
//  * Tiles in bands of four along the tokens, neighbours on one XCD: of its L2 a
//    band shares the weights.  Bands of 1, 2, 4, 8 and 16 take 400, 384, 381, 382
//    and 389 us (gated, 4516 x 12288 x 4096).
// 8192^3 429 us (2560 TFLOP/s; the library's product with one scale for the
// whole operand 459), gated 4516 x 12288 x 4096 380 us (2394), 4096 x 4096 x 12288
// 166 us (2490), 4096 x 8192 x 2560 77 us (2220).
#include "f8.hpp"
#include "f8_device.hpp"
#include "f8_store.hpp"
#include "lds_copy.hpp"

namespace w4a8 {

namespace {

constexpr int LBM = 256, LBN = 256;            // tokens and weight rows of a tile
constexpr int LXB = LBM * 128, LWB = LBN * 128;
constexpr int LSB = LXB + LWB;                 // 64 KiB a stage of 128 bytes of K; two stages

// Workgroup barrier without waits of its own: the kernel waits for its copies
// before it, and what it has read is used before the place is copied over.
__device__ __forceinline__ void stage_barrier()
{
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
}

// At most N of the wave's copies may still be on their way.
template <int N> __device__ __forceinline__ void wait_copies()
{
    __builtin_amdgcn_sched_barrier(0);
    wait_vmcnt<N>();
    __builtin_amdgcn_sched_barrier(0);
}

template <bool GATED, bool TAIL>
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
        // where the tile has no second half the first takes its place, and its
        // columns are not stored: an empty resource would leave it to the range
        // check to sum an offset of K and the lane's without a wrap
        const int n1 = GATED || n0 + 128 >= N ? n0 : n0 + 128;
        rw0 = make_rsrc(a.w[0] + (int64_t)n0 * K, (uint32_t)(min(128, N - n0) * K));
        rw1 = make_rsrc(a.w[GATED] + (int64_t)n1 * K, (uint32_t)(min(128, N - n1) * K));
        const int nb = n0 >> 7, nb1 = n1 >> 7;
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
    // The lane's offsets of the wave's four blocks of x and two of each half of
    // w.  TAIL (128 does not divide K): chunks past the row's end in the last
    // stage read zeros, by an offset past the resource.
    uint32_t xo[4], wo[2], past[2] = {0, 0};
#pragma unroll
    for (int p = 0; p < 4; ++p)
        xo[p] = (uint32_t)((wave * 32 + p * 8 + (lane >> 3)) * K + (chunk0 ^ (16 * (p & 1))));
#pragma unroll
    for (int p = 0; p < 2; ++p)
        wo[p] = (uint32_t)((wave * 16 + p * 8 + (lane >> 3)) * K + (chunk0 ^ (16 * p)));
    if (TAIL)
#pragma unroll
        for (int p = 0; p < 2; ++p)
            past[p] = (chunk0 ^ (16 * p)) >= (K & 127) ? 0x80000000u : 0u;
    auto copy16 = [&](v4i r, uint32_t at, uint32_t offset, int par, int stage) __attribute__((always_inline)) {
        set_m0(at);
        if (TAIL)
            offset |= stage == KB - 1 ? past[par] : 0u;
        copy16_buf_to_lds<0>(r, offset, (uint32_t)(stage * 128));
    };
    auto copy_x = [&](int p) __attribute__((always_inline)) {         // p = 0 .. 3
        copy16(rx, ring_at + cur_buf * LSB + (wave * 4 + p) * 1024, xo[p], p & 1, cur_s);
    };
    auto copy_w0 = [&](int p) __attribute__((always_inline)) {        // p = 0, 1
        copy16(rw0, ring_at + cur_buf * LSB + LXB + (wave * 2 + p) * 1024, wo[p], p, cur_s);
    };
    auto copy_w1 = [&](int p) __attribute__((always_inline)) {        // of the stage before the cursor's
        copy16(rw1_now, ring_at + (cur_buf ^ 1) * LSB + LXB + 16384 + (wave * 2 + p) * 1024, wo[p], p, w1_s);
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
    // stage lane group h takes 0 1, 2 3, 5 4, 7 6.  One LDS address for each of
    // a lane's two chunks, turned to the other buffer each stage; rows and
    // halves are immediate offsets.
    const int lr = lane & 15, lh = lane >> 4;
    const int c0 = lh == 0 ? 0 : lh == 1 ? 2 : lh == 2 ? 5 : 7;
    const int sw8 = (lr & 7) ^ (lr >> 3);
    typedef __attribute__((address_space(3))) const uint8_t lds_bytes;
    typedef __attribute__((address_space(3))) const v4i lds_v4i;
    typedef __attribute__((address_space(3))) const float lds_float;
    uint32_t xa[2], wa[2], sa = scales_at + (uint32_t)(wm * 64 + lr) * 4, ga = scales_at + 1024;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const uint32_t in = (uint32_t)(lr * 128 + 16 * ((c0 ^ q) ^ sw8));
        xa[q] = ring_at + wm * 8192 + in;
        wa[q] = ring_at + LXB + group * 8192 + in;
    }
    auto read16 = [&](uint32_t at, int offset) __attribute__((always_inline)) {
        return *reinterpret_cast<lds_v4i *>(reinterpret_cast<lds_bytes *>(at) + offset);
    };
    auto read_frag = [&](const uint32_t (&at)[2], int offset) __attribute__((always_inline)) {
        return __builtin_shufflevector(read16(at[0], offset), read16(at[1], offset), 0, 1, 2, 3, 4, 5, 6, 7);
    };

    float acc[2][4][4][4];
    v8i xf[4], wf[4];
    v4f pr[4];
    float sc[2][4], sx[4], sw[2];
    auto read_float = [&](uint32_t at, int offset) __attribute__((always_inline)) {
        return *reinterpret_cast<lds_float *>(reinterpret_cast<lds_bytes *>(at) + offset);
    };
    auto read_scales = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            sx[j] = read_float(sa, 64 * j);
        sw[0] = read_float(ga, 0);
        sw[1] = read_float(ga, 256);
    };
    uint32_t to_ring = LSB, to_scales = 2048;         // from this buffer to the other

    // Product t = 0 .. 31 of a stage: half t / 16 of w, its block t / 4 % 4, x's
    // block t % 4.  Each is folded three products later, the last three in the
    // stage that follows.
    auto fold = [&](int u) __attribute__((always_inline)) {
        const int h = u >> 4, i = (u >> 2) & 3, j = u & 3;
#pragma unroll
        for (int r = 0; r < 4; ++r)
            acc[h][i][j][r] = fmaf(pr[j][r], sc[h][j], acc[h][i][j][r]);
    };
    auto half = [&](auto HALF) __attribute__((always_inline)) {
        constexpr int h = decltype(HALF)::value;
#pragma unroll
        for (int q = 0; q < 16; ++q) {
            const int t = 16 * h + q, i = q >> 2, j = q & 3;
            v4f p = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wf[i], xf[j], v4f{0, 0, 0, 0}, 0, 0, 0, 0, 0, 0);
            __builtin_amdgcn_sched_barrier(0);
            fold((t + 29) & 31);
            pr[j] = p;
            // what the products no longer need makes room for what comes next
            if (h == 0) {
                if (j == 3)
                    wf[i] = read_frag(wa, 16384 + 2048 * i);
                if (q == 3) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        sc[1][k] = sx[k] * sw[1];
                }
                if (q == 1 || q == 9)
                    copy_w1(q >> 3);
            } else {
                if (j == 3)
                    wf[i] = read_frag(wa, 2048 * i);
                if (i == 3)
                    xf[j] = read_frag(xa, 2048 * j);
                if (q == 0)
                    read_scales();
                if (q % 2 == 1 && q < 8)
                    copy_x(q >> 1);
                if (q == 9 || q == 11)
                    copy_w0((q - 9) >> 1);
                if (q == 13)
                    copy_scales();
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    // the sums are formed here, not where the compiler next needs them
    auto settle = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
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
    stage_barrier();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        xf[i] = read_frag(xa, 2048 * i);
        wf[i] = read_frag(wa, 2048 * i);
    }
    read_scales();
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
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            pr[j] = v4f{0, 0, 0, 0};
            sc[1][j] = 0.0f;
        }
#pragma clang loop unroll(disable)
        for (int s = 0; s < KB; ++s) {
            wait_copies<7>();                         // this stage's second half of w
            stage_barrier();
            advance();
#pragma unroll
            for (int j = 0; j < 4; ++j)
                sc[0][j] = sx[j] * sw[0];
            half(std::integral_constant<int, 0>());
            wait_copies<2>();                         // the next stage's x, first half of w and scales
            stage_barrier();
            xa[0] += to_ring, xa[1] += to_ring, wa[0] += to_ring, wa[1] += to_ring;
            sa += to_scales, ga += to_scales;
            to_ring = -to_ring, to_scales = -to_scales;
            half(std::integral_constant<int, 1>());
            settle();
        }
        fold(29);
        fold(30);
        fold(31);
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
    const dim3 grid((unsigned)(tiles < a.num_cu ? tiles : a.num_cu));
    if (a.K % 128 == 0)
        hipLaunchKernelGGL((f8_gemm_large_kernel<GATED, false>), grid, dim3(512), 0, st, a, tiles_m, tiles_n, 4);
    else
        hipLaunchKernelGGL((f8_gemm_large_kernel<GATED, true>), grid, dim3(512), 0, st, a, tiles_m, tiles_n, 4);
}

void launch_f8_large(const F8Args &a, bool gated, hipStream_t st)
{
    if (gated)
        launch_large<true>(a, st);
    else
        launch_large<false>(a, st);
}

}  // namespace w4a8

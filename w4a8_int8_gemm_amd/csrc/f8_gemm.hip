// The product in 8-bit floating point with a scale for each block of 128, and
// the gated pair of products of a feed-forward block (gfx950).
//
//     P_b[m, n] = sum over k in block b of x[m, k] w[n, k]        (matrix unit)
//     c[m, n]   = sum_b P_b sx[b, m] sw[n / 128, b]               (fp32)
//     y = fp16(c), or of two such sums y = act(c_gate) c_up, in fp16 or again
//     as e4m3 codes with a scale for each token and 128 columns.
//
// One v_mfma_f32_16x16x128_f8f6f4 is exactly one block b of a 16 x 16 output
// piece, so each instruction starts from zero and its four results a lane go
// into the fp32 sums with one fma each.  The weights are the first operand:
// lane l supplies row l % 16, bytes 32 (l / 16) .. + 31 of both operands, and
// receives token l % 16 of columns 4 (l / 16) .. + 3, so a lane needs one
// scale of x per block and 16 tokens, and stores four columns side by side.
//
// The matrix unit adds a group of eight consecutive products aligned to the
// largest of them and keeps 13 bits below its exponent (measured: a product
// 2^-14 of its group's largest vanishes; groups are then added as fp32).  That
// is part of the hardware's product: relative to sum |x w| an error below
// 8 2^-13, on Gaussian rows 1.4e-5 of the result's size.
#include "f8_few.hpp"
#include "f8_device.hpp"

namespace w4a8 {

namespace {

// 16 bytes of a row at byte k, zeros past the row's end.
__device__ __forceinline__ uint4 row16(const uint8_t *row, int k, int K, bool live)
{
    return live && k < K ? *reinterpret_cast<const uint4 *>(row + k) : make_uint4(0u, 0u, 0u, 0u);
}

__device__ __forceinline__ v8i frag(const uint8_t *row, int k, int K, bool live)
{
    const uint4 a = row16(row, k, K, live), b = row16(row, k + 16, K, live);
    return v8i{(int)a.x, (int)a.y, (int)a.z, (int)a.w, (int)b.x, (int)b.y, (int)b.z, (int)b.w};
}

// 32 tokens x 128 columns a workgroup of four waves, 32 columns each.
template <bool GATED>
__global__ __launch_bounds__(256) void f8_gemm_kernel(F8Args a, int tiles_m, int64_t tiles)
{
    constexpr int SIDES = GATED ? 2 : 1;
    __shared__ uint32_t top[4][32];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int M = a.M, N = a.N, K = a.K;
    const int KB = (K + kF8Block - 1) / kF8Block;
    for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const int nb = (int)(tile / tiles_m);
        const int m0 = (int)(tile % tiles_m) * 32, n0 = nb * 128 + wave * 32;
        v4f acc[SIDES][2][2] = {};
        for (int b = 0; b < KB; ++b) {
            const int k = b * kF8Block + 32 * (lane >> 4);
            v8i xf[2];
            float sx[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int m = m0 + 16 * j + (lane & 15);
                xf[j] = frag(a.x + (int64_t)m * K, k, K, m < M);
                sx[j] = m < M ? a.sx[(int64_t)b * M + m] : 0.0f;
            }
#pragma unroll
            for (int s = 0; s < SIDES; ++s) {
                const float sw = a.sw[s][(int64_t)nb * KB + b];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int n = n0 + 16 * i + (lane & 15);
                    const v8i wf = frag(a.w[s] + (int64_t)n * K, k, K, n < N);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const v4f p = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                            wf, xf[j], v4f{0, 0, 0, 0}, 0, 0, 0, 0, 0, 0);
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            acc[s][i][j][r] = fmaf(p[r], sx[j] * sw, acc[s][i][j][r]);
                    }
                }
            }
        }
        if constexpr (GATED) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        acc[0][i][j][r] = f8_activation(acc[0][i][j][r], a.gelu) * acc[1][i][j][r];
        }
        if (!GATED || a.y) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int m = m0 + 16 * j + (lane & 15);
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int n = n0 + 16 * i + 4 * (lane >> 4) + r;
                        if (m < M && n < N)
                            a.y[(int64_t)m * N + n] = f2h(acc[0][i][j][r]);
                    }
            }
            continue;
        }
        // a token's 128 columns lie in four lanes of each of the four waves
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            uint32_t t = 0;
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    t = max(t, abs_bits(acc[0][i][j][r]));
            t = max(t, (uint32_t)__shfl_xor((int)t, 16));
            t = max(t, (uint32_t)__shfl_xor((int)t, 32));
            if (lane < 16)
                top[wave][16 * j + lane] = t;
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int ml = 16 * j + (lane & 15), m = m0 + ml;
            float s, r;
            f8_block_scale(max(max(top[0][ml], top[1][ml]), max(top[2][ml], top[3][ml])), s, r);
            if (m >= M)
                continue;
            if (wave == 0 && lane < 16)
                a.ys[(int64_t)nb * M + m] = s;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const v4f v = acc[0][i][j];
                const uint32_t c = f8_codes4(v[0], v[1], v[2], v[3], s, r);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int n = n0 + 16 * i + 4 * (lane >> 4) + e;
                    if (n < N)
                        a.yq[(int64_t)m * N + n] = (uint8_t)(c >> (8 * e));
                }
            }
        }
    }
}

}  // namespace

template <bool GATED>
static void launch(const F8Args &a, hipStream_t st)
{
    const int tiles_m = (a.M + 31) / 32;
    const int64_t tiles = (int64_t)tiles_m * ((a.N + 127) / 128);
    const int64_t most = 1 << 20;
    hipLaunchKernelGGL(f8_gemm_kernel<GATED>, dim3((unsigned)(tiles < most ? tiles : most)), dim3(256), 0, st, a,
                       tiles_m, tiles);
}

size_t f8_workspace(int64_t M, int64_t N, int64_t K, bool gated, bool quantize)
{
    return M > 0 && N > 0 && K > 0 && M <= kF8FewTokens ? f8_few_workspace(M, N, K, gated, quantize) : 0;
}

size_t f8_workspace_any(int64_t, int64_t) { return 0; }

void launch_f8(const F8Args &a, bool gated, uint64_t tag, void *workspace, hipStream_t st)
{
    if (a.M <= kF8FewTokens)
        launch_f8_few(a, gated, tag, workspace, st);
    else if (a.M > 64)
        launch_f8_large(a, gated, st);
    else if (gated)
        launch<true>(a, st);
    else
        launch<false>(a, st);
}

}  // namespace w4a8

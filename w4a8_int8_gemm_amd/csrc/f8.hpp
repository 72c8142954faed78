// Launchers of the 8-bit floating point operators (host side).  Arguments are
// validated by the C entry points before any of these is called.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace w4a8 {

// fp16 rows [rows, K] (K % 8 == 0) to e4m3 codes, a scale for each row and
// block of 128: scale [ceil(K / 128), rows].
void launch_quantize_act_f8(const uint16_t *x, int64_t rows, int K, uint8_t *q, float *scale,
                            hipStream_t st);

// fp16 [N, K] to e4m3 codes, a scale for each 128 x 128 block:
// scale [ceil(N / 128), ceil(K / 128)].
void launch_quantize_weight_f8(const uint16_t *w, int64_t N, int K, uint8_t *q, float *scale,
                               hipStream_t st);

// What rmsnorm_quant writes.
enum class NormOut : int { INT8_ROW, INT8_64, INT8_128, F8 };

struct NormArgs {
    const uint16_t *x;          // [M, K]
    const uint16_t *residual;   // [M, K] or null
    const uint16_t *gain;       // [K]
    uint16_t *sum;              // x + residual, [M, K] or null
    uint8_t *q;                 // [M, K] codes
    float *scale;               // [M], [M, K / gs] or, for F8, [ceil(K / 128), M]
    int64_t M;
    int K;
    float eps;
};
void launch_rmsnorm_quant(NormOut out, const NormArgs &a, hipStream_t st);

struct F8Args {
    const uint8_t *x;           // e4m3 [M, K]
    const float *sx;            // [ceil(K / 128), M]
    const uint8_t *w[2];        // e4m3 [N, K]; the second (up) of the gated product only
    const float *sw[2];         // [ceil(N / 128), ceil(K / 128)]
    uint16_t *y;                // fp16 [M, N], or null:
    uint8_t *yq;                // e4m3 [M, N] with
    float *ys;                  // scales [ceil(N / 128), M]
    int M, N, K;
    int gelu;                   // the gated product's activation: 0 silu, 1 gelu (tanh form)
    int num_cu;
};
// The kernel for the sizes: the simple one, for few tokens (with a workspace of
// f8_workspace() bytes and the call's tag among its counters), for large outputs.
size_t f8_workspace(int64_t M, int64_t N, int64_t K, bool gated, bool quantize);
size_t f8_workspace_any(int64_t M, int64_t K);     // a product's, not gated, for every N
void launch_f8(const F8Args &a, bool gated, uint64_t tag, void *workspace, hipStream_t st);
void launch_f8_few(const F8Args &a, bool gated, uint64_t tag, void *workspace, hipStream_t st);
void launch_f8_large(const F8Args &a, bool gated, hipStream_t st);

}  // namespace w4a8

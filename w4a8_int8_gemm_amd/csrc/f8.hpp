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
    float lift, unlift;         // the launcher's (norm_inverse)
};
void launch_rmsnorm_quant(NormOut out, NormArgs a, hipStream_t st);

struct F8Args {
    const uint8_t *x;           // e4m3 [M, K]
    const float *sx;            // [ceil(K / 128)] rows of M scales, sm apart
    const uint8_t *w[2];        // e4m3 [N, K]; the second (up) of the gated product only
    const float *sw[2];         // [ceil(N / 128), ceil(K / 128)]
    uint16_t *y;                // fp16, rows of N values yn apart, or null:
    uint8_t *yq;                // e4m3, likewise, with
    float *ys;                  // scales [ceil(N / 128)] rows of M, sm apart
    int M, N, K;
    int sm, yn;                 // M and N of the whole call, of which this may be a part
    int gelu;                   // the gated product's activation: 0 silu, 1 gelu (tanh form)
    int num_cu;
};

// What several workgroups of one launch leave for the last of them: the sums of
// 128 columns, or (f8_tile.hip with K in parts) those of a tile.
struct F8Parts {
    int splits;                 // ranges of K
    uint64_t tag;               // of the call among the counters
    uint64_t *counters;         // one for each 128 columns or tile, kCounterStride apart
    float *sums;                // [ceil(N / 128)][splits][M][128], or [splits][tiles][sums of a tile]
};

// Bytes of workspace (f8_plan.hip); the product on checked arguments, by the
// kernels that suit its sizes.
size_t f8_workspace(int64_t M, int64_t N, int64_t K, bool gated, bool quantize);
size_t f8_workspace_any(int64_t M, int64_t K);     // the largest of a product's, not gated, over all N
void launch_f8(const F8Args &a, bool gated, uint64_t tag, void *workspace, hipStream_t st);

// The kernels.  Few tokens: at most kF8FewTokens.  Tiles: kF8Tiles' shapes.
constexpr int kF8FewTokens = 64;
void launch_f8_few(const F8Args &a, bool gated, const F8Parts &f, hipStream_t st);
struct F8Tile {
    int tokens, columns;
};
constexpr int kF8TileShapes = 5;
constexpr F8Tile kF8Tiles[kF8TileShapes] = {{64, 64}, {64, 128}, {96, 128}, {128, 64}, {128, 128}};
void launch_f8_tile(const F8Args &a, bool gated, int shape, const F8Parts &f, hipStream_t st);
void launch_f8_large(const F8Args &a, bool gated, hipStream_t st);

}  // namespace w4a8

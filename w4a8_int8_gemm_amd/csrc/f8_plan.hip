// Which kernels a product in 8-bit floating point runs with, by its sizes.
#include "f8.hpp"
#include "kv4.hpp"

namespace w4a8 {

namespace {

// Ranges of K in the kernel for few tokens: where 16 columns a workgroup leave
// three quarters of the chip idle, K is cut in up to four.  64 x 1024 x 14336
// 14.5 us in one range, 11.1 in four; 1 x 256 x 14336 7.1 and 6.0; but 1 x 2560
// x 10240 8.1 in one, 10.0 in two: the parts' meeting takes 3 to 4 us.
int few_splits(int64_t N, int64_t K, bool gated)
{
    const int64_t groups = (N + 15) / 16, blocks = (K + 127) / 128;
    if (gated || groups > 64 || blocks < 64)
        return 1;
    return groups > 32 ? 2 : 4;
}

bool few(int64_t M, int64_t N)
{
    // Above 32 tokens each workgroup's copy of x outweighs its weights: 64 x 64
    // tiles read it a quarter as often, once there are enough of them.  64
    // tokens: 64 tiles (4096 columns, K 4096) 12.0 us against 8.0 here, 160
    // (10240, 2560) 13.3 against 16.8, 448 (28672, 4096) 31.8 against 50.
    return M <= 32 || (M <= kF8FewTokens && (N + 63) / 64 < 128);
}

size_t counter_bytes(int64_t N) { return kv4_counter_bytes((N + 127) / 128, 1); }

int splits_of(int64_t M, int64_t N, int64_t K, bool gated)
{
    return few(M, N) ? few_splits(N, K, gated) : 1;
}

// Microseconds, as a model: kernels for one to 256 tokens take the time of their
// copies into LDS, 14.1 ns for one of 1 KiB by a workgroup that has a compute
// unit of its own (16.3 where two share one), or of the stages on the way;
// a stage of a large tile takes 0.96 to 1.1 us with the share of the chip that
// is busy.  Fitted to 128 shapes (65 to 3000 tokens, 1024 to 14336 columns and
// K, weights from HBM) with every kernel: the choice is 0.4 % slower than the
// best on average, 8 % at most.
constexpr double kStart = 5.5;
constexpr double kMeet = 3.0, kMeetByte = 1.5e-5;       // parts of K: their meeting, and each byte of a part's sums
constexpr double kSecond = 2.0;         // what of it a second launch right behind the first does not take

// A stage of a workgroup where each has a compute unit of its own.
double stage_time(int shape, bool gated, int64_t groups, int num_cu)
{
    const F8Tile t = kF8Tiles[shape];
    const int copies = (t.tokens + (gated ? 2 : 1) * t.columns) / 8 + 4;
    const int stage = (t.tokens + (gated ? 2 : 1) * t.columns) * 128 + 1024;
    const int all = 157 * 1024 / stage, deep = all < 8 ? all : 8;
    const double alone = 0.0141 * copies, wait = 0.97 / (deep - 1) * (0.5 + 0.5 * (double)groups / num_cu);
    return alone > wait ? alone : wait;
}

double tile_time(int shape, int64_t M, int64_t N, int64_t K, bool gated, int num_cu)
{
    const F8Tile t = kF8Tiles[shape];
    const int64_t stages = (K + 127) / 128;
    const int64_t groups = ((M + t.tokens - 1) / t.tokens) * ((N + t.columns - 1) / t.columns);
    const int copies = (t.tokens + (gated ? 2 : 1) * t.columns) / 8 + 4;
    const int stage = (t.tokens + (gated ? 2 : 1) * t.columns) * 128 + 1024;
    const int all = 157 * 1024 / stage, half = 78 * 1024 / stage;
    const int deep = all < 8 ? all : 8;
    const double alone = 0.0141 * copies, wait = 0.97 / (deep - 1);
    if (groups <= num_cu)
        return kStart + stages * stage_time(shape, gated, groups, num_cu);
    if (half < 2)
        return kStart + stages * (alone > wait ? alone : wait) * ((groups + num_cu - 1) / num_cu);
    const double two = 2 * 0.0163 * copies;
    const int64_t rest = groups % (2 * num_cu);
    return kStart + stages * ((groups / (2 * num_cu)) * two + (rest > num_cu ? 0.9 * two : rest > 0 ? alone : 0.0));
}

double large_time(int64_t M, int64_t N, int64_t K, bool gated, int num_cu)
{
    const int64_t tiles = ((M + 255) / 256) * ((N + (gated ? 127 : 255)) / (gated ? 128 : 256));
    const int64_t rounds = (tiles + num_cu - 1) / num_cu;
    return kStart + rounds * (((K + 127) / 128) * (0.96 + 0.15 * (double)tiles / ((double)num_cu * rounds)) + 2.7);
}

// The best tile shape, or kF8TileShapes for the large kernel.
int best_shape(int64_t M, int64_t N, int64_t K, bool gated, bool quantize, int num_cu, double *time)
{
    int best = kF8TileShapes;
    *time = large_time(M, N, K, gated, num_cu);
    for (int i = 0; i < kF8TileShapes; ++i) {
        // e4m3 output: a workgroup holds the 128 columns of a scale (64 tokens
        // and fewer can meet in the workspace)
        if (quantize && kF8Tiles[i].columns < 128)
            continue;
        // a launch of 2^32 threads would wrap
        if (((M + 63) / 64) * ((N + 63) / 64) >= (1 << 24))
            continue;
        const double t = tile_time(i, M, N, K, gated, num_cu);
        if (t < *time) {
            *time = t;
            best = i;
        }
    }
    return best;
}

// Where more than 64 tokens' tiles leave half of the chip idle or more, K in
// `splits` parts, a workgroup each, that meet in the workspace, if the model
// says so: 128 x 4096 x 14336 37.8 us in one part, 24.5 in four; 111 x 776 x 6880
// 18.8 and 10.9; 1272 x 183 x 10224 28.2 and 15.3; but 303 x 2991 x 5520 18.1 in
// one.  Parts under eight stages are not worth their start.  Of the sizes
// alone, as the workspace is, for the 256 compute units of the chip.
struct Cut {
    int shape, splits;
    int64_t tiles;
    size_t bytes;                                          // of one part's sums
};
constexpr int kCutCUs = 256;

Cut cut_of(int64_t M, int64_t N, int64_t K, bool gated, bool quantize)
{
    Cut best = {0, 1, 0, 0};
    const int64_t blocks = (K + 127) / 128;
    if (M <= kF8FewTokens || blocks < 16 || (M + 127) / 128 > kCutCUs / 2 || (N + 127) / 128 > kCutCUs / 2)
        return best;
    double time;
    best_shape(M, N, K, gated, quantize, kCutCUs, &time);
    for (int i = 0; i < kF8TileShapes; ++i) {
        const F8Tile t = kF8Tiles[i];
        if (quantize && t.columns < 128)
            continue;
        const int64_t tiles = ((M + t.tokens - 1) / t.tokens) * ((N + t.columns - 1) / t.columns);
        const int64_t size = (gated ? 2 : 1) * t.tokens * t.columns * (int)sizeof(float);      // of a part's sums of a tile
        for (int s = 2; s <= 8 && s * tiles <= kCutCUs && blocks / s >= 8; ++s) {
            const double cut = kStart + (double)((blocks + s - 1) / s) * stage_time(i, gated, s * tiles, kCutCUs) +
                               kMeet + (s + 1) * (double)size * kMeetByte;
            if (cut < time) {
                time = cut;
                best = {i, s, tiles, (size_t)(tiles * size)};
            }
        }
    }
    return best;
}

void launch_shape(const F8Args &a, bool gated, int shape, const F8Parts &f, hipStream_t st)
{
    if (shape < kF8TileShapes)
        launch_f8_tile(a, gated, shape, f, st);
    else
        launch_f8_large(a, gated, st);
}

}  // namespace

size_t f8_workspace(int64_t M, int64_t N, int64_t K, bool gated, bool quantize)
{
    if (M <= 0 || N <= 0 || K <= 0)
        return 0;
    if (M > kF8FewTokens) {
        const Cut c = cut_of(M, N, K, gated, quantize);
        return c.splits == 1 ? 0 : kv4_counter_bytes(c.tiles, 1) + c.splits * c.bytes;
    }
    const int splits = splits_of(M, N, K, gated);
    if (splits == 1 && !quantize)
        return 0;
    return counter_bytes(N) + (size_t)((N + 127) / 128) * splits * (size_t)M * 128 * sizeof(float);
}

size_t f8_workspace_any(int64_t M, int64_t K)
{
    if (M > kF8FewTokens)                          // at most as many 128 x 128 tiles as compute units
        return (K + 127) / 128 < 16 || (M + 127) / 128 > kCutCUs / 2
                   ? 0
                   : kv4_counter_bytes(kCutCUs, 1) + (size_t)kCutCUs * 128 * 128 * sizeof(float);
    size_t most = 0;
    for (int64_t N : {512, 1024})                  // the widest outputs cut in four and in two
        most = f8_workspace(M, N, K, false, false) > most ? f8_workspace(M, N, K, false, false) : most;
    return most;
}

void launch_f8(const F8Args &a, bool gated, uint64_t tag, void *workspace, hipStream_t st)
{
    const bool quantize = gated && !a.y;
    F8Parts f;
    f.splits = splits_of(a.M, a.N, a.K, gated);
    f.tag = tag;
    f.counters = static_cast<uint64_t *>(workspace);
    f.sums = reinterpret_cast<float *>(static_cast<char *>(workspace) + counter_bytes(a.N));
    if (few(a.M, a.N)) {
        launch_f8_few(a, gated, f, st);
        return;
    }
    if (a.M <= kF8FewTokens) {
        launch_f8_tile(a, gated, 0, f, st);
        return;
    }
    const Cut cut = cut_of(a.M, a.N, a.K, gated, quantize);
    if (cut.splits > 1) {
        f.splits = cut.splits;
        f.sums = reinterpret_cast<float *>(static_cast<char *>(workspace) + kv4_counter_bytes(cut.tiles, 1));
        launch_f8_tile(a, gated, cut.shape, f, st);
        return;
    }
    // Whole rounds of large tiles over the chip, and what is left of the tokens
    // or of the columns by the kernel that suits it, where that is faster than
    // a last round that leaves most of the chip idle.
    double time;
    const int shape = best_shape(a.M, a.N, a.K, gated, quantize, a.num_cu, &time);
    const int columns = gated ? 128 : 256;
    const int64_t tm = (a.M + 255) / 256, tn = (a.N + columns - 1) / columns;
    int64_t best_m = 0, best_n = 0;
    int best_rest = 0;
    for (int64_t rounds = tm * tn / a.num_cu; rounds > 0 && rounds >= tm * tn / a.num_cu - 1; --rounds) {
        const int64_t rows = rounds * a.num_cu / tn, cols = rounds * a.num_cu / tm;
        double rest;
        if (rows > 0 && rows < tm) {
            const int s = best_shape(a.M - 256 * rows, a.N, a.K, gated, quantize, a.num_cu, &rest);
            rest += large_time(256 * rows, a.N, a.K, gated, a.num_cu) - kSecond;
            if (rest < time) {
                time = rest;
                best_m = 256 * rows, best_n = 0, best_rest = s;
            }
        }
        if (cols > 0 && cols < tn) {
            const int s = best_shape(a.M, a.N - columns * cols, a.K, gated, quantize, a.num_cu, &rest);
            rest += large_time(a.M, columns * cols, a.K, gated, a.num_cu) - kSecond;
            if (rest < time) {
                time = rest;
                best_m = 0, best_n = columns * cols, best_rest = s;
            }
        }
    }
    if (best_m + best_n == 0) {
        launch_shape(a, gated, shape, f, st);
        return;
    }
    F8Args first = a, second = a;
    if (best_m > 0) {
        first.M = (int)best_m;
        second.M = (int)(a.M - best_m);
        second.x += best_m * a.K;
        second.sx += best_m;
        if (a.y)
            second.y += best_m * a.yn;
        else
            second.yq += best_m * a.yn, second.ys += best_m;
    } else {
        first.N = (int)best_n;
        second.N = (int)(a.N - best_n);
        for (int i = 0; i < (gated ? 2 : 1); ++i) {
            second.w[i] += best_n * a.K;
            second.sw[i] += best_n / 128 * ((a.K + 127) / 128);
        }
        if (a.y)
            second.y += best_n;
        else
            second.yq += best_n, second.ys += best_n / 128 * a.sm;
    }
    launch_f8_large(first, gated, st);
    launch_shape(second, gated, best_rest, f, st);
}

}  // namespace w4a8

// Host build of the 8-bit floating point products' choice of kernels (w4a8_int8_gemm_amd/csrc/f8_plan.hip)
// with launches that only write down what they were asked for.  Test code only.
#include <vector>

#include "../../w4a8_int8_gemm_amd/csrc/f8_plan.hip"

namespace {
struct Launch {
    int64_t kind, shape, splits, m0, n0, M, N, side;
};
std::vector<Launch> made;
w4a8::F8Args whole;

// where the launch begins in the whole product, by its pointers; -1 where they do not agree
void note(const w4a8::F8Args &a, bool gated, int kind, int shape, int splits)
{
    Launch l = {kind, shape, splits, 0, 0, a.M, a.N, gated ? 2 : 1};
    const int64_t K = a.K, KB = (K + 127) / 128;
    l.m0 = (a.x - whole.x) / K;
    l.n0 = (a.w[0] - whole.w[0]) / K;
    bool same = a.x == whole.x + l.m0 * K && a.sx == whole.sx + l.m0 && a.sm == whole.sm && a.yn == whole.yn &&
                a.K == whole.K && a.gelu == whole.gelu && a.num_cu == whole.num_cu && l.n0 % 128 == 0;
    for (int i = 0; i < (gated ? 2 : 1); ++i)
        same = same && a.w[i] == whole.w[i] + l.n0 * K && a.sw[i] == whole.sw[i] + l.n0 / 128 * KB;
    if (whole.y)
        same = same && a.y == whole.y + l.m0 * a.yn + l.n0;
    else
        same = same && !a.y && a.yq == whole.yq + l.m0 * a.yn + l.n0 && a.ys == whole.ys + l.n0 / 128 * a.sm + l.m0;
    if (!same)
        l.m0 = -1;
    made.push_back(l);
}
}  // namespace

namespace w4a8 {
void launch_f8_few(const F8Args &a, bool gated, const F8Parts &f, hipStream_t) { note(a, gated, 0, 0, f.splits); }
void launch_f8_tile(const F8Args &a, bool gated, int shape, const F8Parts &f, hipStream_t) { note(a, gated, 1, shape, f.splits); }
void launch_f8_large(const F8Args &a, bool gated, hipStream_t) { note(a, gated, 2, 0, 1); }
}  // namespace w4a8

extern "C" {

// out: up to 4 launches of 8 numbers; returns their count.  Addresses are only compared, never read.
int shim_plan(int M, int N, int K, int gated, int quantize, int num_cu, int64_t *out)
{
    using namespace w4a8;
    F8Args a = {};
    const auto at = [](int64_t i) { return reinterpret_cast<char *>((intptr_t)i << 56); };
    a.x = (const uint8_t *)at(1), a.sx = (const float *)at(2);
    for (int i = 0; i < 2; ++i)
        a.w[i] = (const uint8_t *)at(3 + i), a.sw[i] = (const float *)at(5 + i);
    if (quantize)
        a.yq = (uint8_t *)at(7), a.ys = (float *)at(8);
    else
        a.y = (uint16_t *)at(9);
    a.M = a.sm = M, a.N = a.yn = N, a.K = K, a.num_cu = num_cu;
    whole = a;
    made.clear();
    launch_f8(a, gated != 0, 5, nullptr, nullptr);
    const int n = (int)made.size() < 4 ? (int)made.size() : 4;
    for (int i = 0; i < n; ++i) {
        const Launch &l = made[i];
        const int64_t v[8] = {l.kind, l.shape, l.splits, l.m0, l.n0, l.M, l.N, l.side};
        for (int j = 0; j < 8; ++j)
            out[8 * i + j] = v[j];
    }
    return (int)made.size();
}

int64_t shim_workspace(int64_t M, int64_t N, int64_t K, int gated, int quantize)
{
    return (int64_t)w4a8::f8_workspace(M, N, K, gated != 0, quantize != 0);
}

int64_t shim_workspace_any(int64_t M, int64_t K) { return (int64_t)w4a8::f8_workspace_any(M, K); }

}

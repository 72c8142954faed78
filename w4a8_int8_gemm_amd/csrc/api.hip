// C entry points of libw4a8: argument checks, device check, kernel dispatch.
// The operations and their sources are described in include/w4a8.h.
#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include <time.h>
#include <unistd.h>

#include <atomic>

#include "../../include/w4a8.h"
#include "f8.hpp"
#include "kernels.hpp"
#include "kv4.hpp"

using namespace w4a8;

namespace {

thread_local char g_err[512] = "";

w4a8_status_t fail(w4a8_status_t st, const char *fmt, ...)
{
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_err, sizeof g_err, fmt, ap);
    va_end(ap);
    return st;
}

w4a8_status_t ok()
{
    g_err[0] = '\0';
    return W4A8_OK;
}

constexpr int64_t kMaxDim = 0x7fffffff;
constexpr int64_t kMaxKPerChannel = 133144;   // largest K with 127^2 * K < 2^31
constexpr int64_t kMaxKMv = 32768;            // the token's codes are staged in LDS
constexpr int64_t kMaxKWoMv = 16384;          // weight-only decode: the token as fp32 in LDS
constexpr int64_t kMaxKGemm = int64_t(1) << 22; // a 256-row tile of K bytes stays below 2^30
constexpr int64_t kMaxTiles = 0x7fffffff;     // 32 x 128 output tiles
// Few-token per-channel and W4A8 products (the weight rows streamed whole): up
// to 4 tokens, whose codes are staged in LDS
constexpr int64_t kMaxMFew = 4;
constexpr int64_t kMaxFewCodes = 65536;       // M * K bytes

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned8(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }
bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Per device ordinal: its compute-unit count if it is a gfx950, 0 if it is
// something else, -1 while not yet known.
std::atomic<int> g_dev_cu[64];
struct DevInit {
    DevInit() { for (auto &a : g_dev_cu) a.store(-1); }
} g_dev_init;

// The current device must be a gfx950; *num_cu receives its compute units.
w4a8_status_t check_device(int *num_cu = nullptr)
{
    int dev = -1;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess || dev < 0)
        return fail(W4A8_ERR_DEVICE, "no HIP device (%s)", hipGetErrorString(e));
    if (dev < 64) {
        const int known = g_dev_cu[dev].load(std::memory_order_relaxed);
        if (known > 0) {
            if (num_cu)
                *num_cu = known;
            return W4A8_OK;
        }
        if (known == 0)
            return fail(W4A8_ERR_DEVICE, "HIP device %d is not gfx950", dev);
    }
    hipDeviceProp_t prop;
    e = hipGetDeviceProperties(&prop, dev);
    if (e != hipSuccess)
        return fail(W4A8_ERR_DEVICE, "hipGetDeviceProperties failed: %s", hipGetErrorString(e));
    const bool is950 = strncmp(prop.gcnArchName, "gfx950", 6) == 0;
    const int cus = prop.multiProcessorCount > 0 ? prop.multiProcessorCount : 1;
    if (dev < 64)
        g_dev_cu[dev].store(is950 ? cus : 0, std::memory_order_relaxed);
    if (!is950)
        return fail(W4A8_ERR_DEVICE, "HIP device %d is %s, not gfx950", dev, prop.gcnArchName);
    if (num_cu)
        *num_cu = cus;
    return W4A8_OK;
}

w4a8_status_t check_launch(const char *what)
{
    hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return fail(W4A8_ERR_LAUNCH, "%s: launch failed: %s", what, hipGetErrorString(e));
    return ok();
}

// ---- argument checks (no HIP calls)

w4a8_status_t check_quant(const char *fn, const void *x, int64_t rows, int64_t K, int32_t gs,
                          const void *q, const float *scale, bool int4)
{
    if (rows < 0 || K < 0 || rows > kMaxDim || K > kMaxDim)
        return fail(W4A8_ERR_INVALID_ARG, "%s: sizes out of range (rows=%lld K=%lld)", fn,
                    (long long)rows, (long long)K);
    if (K == 0 || K % 8 != 0)
        return fail(W4A8_ERR_SHAPE, "%s: K=%lld must be a positive multiple of 8", fn, (long long)K);
    if (int4 ? !(gs == 64 || gs == 128) : !(gs == 0 || gs == 64 || gs == 128))
        return fail(W4A8_ERR_SHAPE, "%s: group_size=%d not supported", fn, gs);
    if (gs > 0 && K % gs != 0)
        return fail(W4A8_ERR_SHAPE, "%s: K=%lld is not a multiple of group_size=%d", fn,
                    (long long)K, gs);
    if (rows == 0)
        return W4A8_OK;
    if (!x || !q || !scale)
        return fail(W4A8_ERR_INVALID_ARG, "%s: null pointer", fn);
    if (!aligned16(x) || !aligned16(q) || !aligned4(scale))
        return fail(W4A8_ERR_ALIGNMENT, "%s: tensors must be 16-byte aligned", fn);
    return W4A8_OK;
}

w4a8_status_t check_gemm(const char *fn, const void *xq, const void *w, const void *out,
                         const float *sa, const float *sw, int64_t M, int64_t N, int64_t K,
                         int32_t gs, bool pergroup, bool need_scales)
{
    if (M < 0 || N < 0 || K < 0 || M > kMaxDim || N > kMaxDim || K > kMaxDim)
        return fail(W4A8_ERR_INVALID_ARG, "%s: sizes out of range (M=%lld N=%lld K=%lld)", fn,
                    (long long)M, (long long)N, (long long)K);
    if (K == 0 || K % 64 != 0)
        return fail(W4A8_ERR_SHAPE, "%s: K=%lld must be a positive multiple of 64", fn,
                    (long long)K);
    if (pergroup) {
        if (!(gs == 64 || gs == 128))
            return fail(W4A8_ERR_SHAPE, "%s: group_size=%d must be 64 or 128", fn, gs);
        if (K % gs != 0)
            return fail(W4A8_ERR_SHAPE, "%s: K=%lld is not a multiple of group_size=%d", fn,
                        (long long)K, gs);
    } else if (K > kMaxKPerChannel) {
        return fail(W4A8_ERR_SHAPE, "%s: K=%lld could overflow the int32 sums (max %lld)", fn,
                    (long long)K, (long long)kMaxKPerChannel);
    }
    if (K > kMaxKGemm)
        return fail(W4A8_ERR_SHAPE, "%s: K=%lld exceeds %lld", fn, (long long)K,
                    (long long)kMaxKGemm);
    if (((M + 31) / 32) * ((N + 127) / 128) > kMaxTiles)
        return fail(W4A8_ERR_SHAPE, "%s: output of %lld x %lld is too large", fn, (long long)M,
                    (long long)N);
    if (M == 0 || N == 0)
        return W4A8_OK;
    if (!xq || !w || !out || (need_scales && (!sa || !sw)))
        return fail(W4A8_ERR_INVALID_ARG, "%s: null pointer", fn);
    if (!aligned16(xq) || !aligned16(w) || !aligned16(out) ||
        (need_scales && (!aligned4(sa) || !aligned4(sw))))
        return fail(W4A8_ERR_ALIGNMENT, "%s: tensors must be 16-byte aligned", fn);
    return W4A8_OK;
}

w4a8_status_t check_mv(const void *x, const void *w, const float *sw, const void *y, int64_t N,
                       int64_t K, const int8_t *xq_out, const float *xs_out)
{
    if (N < 0 || K < 0 || N > kMaxDim)
        return fail(W4A8_ERR_INVALID_ARG, "int8_mv: sizes out of range");
    if (K == 0 || K % 16 != 0 || K > kMaxKMv)
        return fail(W4A8_ERR_SHAPE, "int8_mv: K=%lld must be a multiple of 16 in (0, %lld]",
                    (long long)K, (long long)kMaxKMv);
    if (!x)
        return fail(W4A8_ERR_INVALID_ARG, "int8_mv: null x");
    if (N > 0 && (!w || !sw || !y))
        return fail(W4A8_ERR_INVALID_ARG, "int8_mv: null pointer");
    if (!aligned16(x) || (N > 0 && (!aligned16(w) || !aligned4(sw) || !aligned4(y))) ||
        (xq_out && !aligned16(xq_out)) || (xs_out && !aligned4(xs_out)))
        return fail(W4A8_ERR_ALIGNMENT, "int8_mv: misaligned tensor");
    return W4A8_OK;
}

w4a8_status_t check_mv_group(const char *fn, const void *x, const void *w, const float *sw,
                             const void *y, int64_t N, int64_t K, int32_t gs)
{
    if (N < 0 || K < 0 || N > kMaxDim)
        return fail(W4A8_ERR_INVALID_ARG, "%s: sizes out of range", fn);
    if (gs != 64 && gs != 128)
        return fail(W4A8_ERR_SHAPE, "%s: group_size %d must be 64 or 128", fn, (int)gs);
    if (K == 0 || K % 64 != 0 || K % gs != 0 || K > kMaxKMv)
        return fail(W4A8_ERR_SHAPE, "%s: K=%lld must be a multiple of 64 and of group_size in "
                    "(0, %lld]", fn, (long long)K, (long long)kMaxKMv);
    if (!x || (N > 0 && (!w || !sw || !y)))
        return fail(W4A8_ERR_INVALID_ARG, "%s: null pointer", fn);
    if (!aligned16(x) || (N > 0 && (!aligned16(w) || !aligned4(sw) || !aligned4(y))))
        return fail(W4A8_ERR_ALIGNMENT, "%s: misaligned tensor", fn);
    return W4A8_OK;
}

size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

// A tag per call for the counters in its workspace: 48 bits
// over a 16-bit count, other than those of the calls before and, by a start
// from the clock, the process and where it lies, of other processes'.  (No
// std::random_device: it may throw, and this is behind a C entry point.)
uint64_t first_tag()
{
    struct timespec now = {0, 0};
    clock_gettime(CLOCK_REALTIME, &now);
    const uint64_t x = ((uint64_t)now.tv_sec * 1000000000u + (uint64_t)now.tv_nsec) ^ ((uint64_t)getpid() << 32) ^
                       (uint64_t)reinterpret_cast<uintptr_t>(&now);
    return (x * 0x9e3779b97f4a7c15u) >> 17;              // 2^64 over the golden ratio: every bit reaches the upper ones
}

uint64_t next_tag()
{
    static std::atomic<uint64_t> tag{first_tag()};
    return (tag.fetch_add(1, std::memory_order_relaxed) | (uint64_t(1) << 47)) << 16;
}

// ---- 8-bit floating point

constexpr int64_t kMaxRowsF8 = int64_t(1) << 25;   // rows a launch of one wavefront each can number
constexpr int64_t kMaxColumnsF8 = int64_t(1) << 27; // columns a launch of 256 threads for 16 can

// The sizes and buffers of a product's operands: x (codes, or fp16 of the
// same alignment) with or without scales, one or two weights.
w4a8_status_t check_f8(const char *fn, const void *x, const float *sx, bool need_sx, const void *w,
                       const float *sw, const void *w2, const float *sw2, bool gated, int64_t M,
                       int64_t N, int64_t K)
{
    if (M < 0 || N < 0 || K < 0 || M > kMaxRowsF8 || N > kMaxColumnsF8)
        return fail(W4A8_ERR_INVALID_ARG, "%s: sizes out of range (M=%lld N=%lld K=%lld)", fn,
                    (long long)M, (long long)N, (long long)K);
    if (K == 0 || K % 16 != 0 || K > kMaxKGemm)
        return fail(W4A8_ERR_SHAPE, "%s: K=%lld must be a positive multiple of 16 up to %lld", fn,
                    (long long)K, (long long)kMaxKGemm);
    if (((M + 31) / 32) * ((N + 127) / 128) > kMaxTiles)
        return fail(W4A8_ERR_SHAPE, "%s: output of %lld x %lld is too large", fn, (long long)M,
                    (long long)N);
    if (M == 0 || N == 0)
        return W4A8_OK;
    if (!x || !w || !sw || (need_sx && !sx) || (gated && (!w2 || !sw2)))
        return fail(W4A8_ERR_INVALID_ARG, "%s: null pointer", fn);
    if (!aligned16(x) || !aligned16(w) || !aligned16(w2) || !aligned4(sx) || !aligned4(sw) ||
        !aligned4(sw2))
        return fail(W4A8_ERR_ALIGNMENT, "%s: tensors must be 16-byte aligned", fn);
    return W4A8_OK;
}

w4a8_status_t check_workspace(const char *fn, size_t need, const void *workspace, size_t bytes)
{
    if (need > 0 && (!workspace || bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0))
        return fail(W4A8_ERR_WORKSPACE, "%s: workspace of %zu bytes (256-byte aligned) needed, got %zu",
                    fn, need, bytes);
    return W4A8_OK;
}

F8Args make_f8(const uint8_t *x, const float *sx, const uint8_t *w, const float *sw, const uint8_t *w2,
               const float *sw2, int64_t M, int64_t N, int64_t K)
{
    F8Args a{};
    a.x = x; a.sx = sx;
    a.w[0] = w; a.sw[0] = sw; a.w[1] = w2; a.sw[1] = sw2;
    a.M = a.sm = (int)M; a.N = a.yn = (int)N; a.K = (int)K;
    return a;
}

// The product on checked arguments.
w4a8_status_t run_f8(const char *fn, F8Args a, bool gated, void *workspace, w4a8_stream_t stream)
{
    w4a8_status_t st = check_device(&a.num_cu);
    if (st != W4A8_OK)
        return st;
    launch_f8(a, gated, next_tag(), workspace, (hipStream_t)stream);
    return check_launch(fn);
}

// linear()'s workspace in the F8 mode: codes, scales, and what the product
// needs, of N columns or (N < 0: the query does not know N) of any.
struct F8Linear {
    size_t codes, scales, product;
    F8Linear(int64_t M, int64_t K, int64_t N = -1)
        : codes(align256((size_t)M * (size_t)K)),
          scales(align256((size_t)M * (size_t)((K + 127) / 128) * sizeof(float))),
          product(N < 0 ? f8_workspace_any(M, K) : f8_workspace(M, N, K, false, false)) {}
    size_t bytes() const { return codes + scales + product; }
};

// ---- the static scratch of linear_noalloc(): the activations' codes and
// fp32 scales, and in the F8 mode what its product needs, live in this device
// array instead of a caller workspace.
// Each device the library runs on holds its own copy (placed when the code
// object is loaded there) until the process ends.  Host code never passes
// the array's name to a kernel (on the host it only names the symbol): the
// device address is looked up per device with hipGetSymbolAddress and kept.
constexpr size_t kScratchBytes = size_t(64) << 20;
static __device__ __align__(256) uint8_t scratch[kScratchBytes];
std::atomic<uintptr_t> g_scratch_dev[64];     // per device ordinal; 0 = not looked up yet

// Device address of the current device's copy of `scratch`.
w4a8_status_t scratch_address(void **out)
{
    int dev = -1;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess || dev < 0 || dev >= 64)
        return fail(W4A8_ERR_DEVICE, "no HIP device for the static scratch (%s)",
                    hipGetErrorString(e));
    uintptr_t p = g_scratch_dev[dev].load(std::memory_order_acquire);
    if (p == 0) {
        void *ptr = nullptr;
        e = hipGetSymbolAddress(&ptr, HIP_SYMBOL(scratch));
        if (e != hipSuccess || ptr == nullptr)
            return fail(W4A8_ERR_DEVICE, "hipGetSymbolAddress(scratch) on device %d failed: %s",
                        dev, hipGetErrorString(e));
        p = reinterpret_cast<uintptr_t>(ptr);
        g_scratch_dev[dev].store(p, std::memory_order_release);
    }
    *out = reinterpret_cast<void *>(p);
    return W4A8_OK;
}

GemmArgs make_args(const int8_t *xq, const float *sa, const void *w, const float *sw, void *out,
                   int64_t M, int64_t N, int64_t K, int gs)
{
    GemmArgs a;
    a.xq = xq; a.sa = sa; a.w = w; a.sw = sw; a.out = out;
    a.M = (int)M; a.N = (int)N; a.K = (int)K; a.gs = gs;
    a.num_cu = 1;
    return a;
}

w4a8_status_t run_gemm(const char *fn, GemmMode mode, const GemmArgs &a, w4a8_stream_t stream)
{
    if (a.M == 0 || a.N == 0)
        return ok();
    GemmArgs la = a;
    w4a8_status_t st = check_device(&la.num_cu);
    if (st != W4A8_OK)
        return st;
    launch_gemm(mode, la, (hipStream_t)stream);
    return check_launch(fn);
}

// The per-channel product on checked arguments: up to four tokens as the
// few-token matrix-vector form (same arithmetic), else the GEMM.
w4a8_status_t run_pc(const char *fn, const int8_t *xq, const float *xs, const int8_t *wq,
                     const float *sw, w4a8_f16 *y, int64_t M, int64_t N, int64_t K,
                     w4a8_stream_t stream)
{
    if (M >= 1 && M <= kMaxMFew && M * K <= kMaxFewCodes) {
        if (N == 0)
            return ok();
        w4a8_status_t st = check_device();
        if (st != W4A8_OK)
            return st;
        launch_few_pc(xq, xs, wq, sw, y, (int)M, (int)N, (int)K, (hipStream_t)stream);
        return check_launch(fn);
    }
    return run_gemm(fn, GemmMode::PC, make_args(xq, xs, wq, sw, y, M, N, K, 0), stream);
}

// The W4A8 product on checked arguments: up to four tokens as the few-token
// matrix-vector form, else the GEMM.
w4a8_status_t run_w4(const char *fn, const int8_t *xq, const float *xs, const uint8_t *w4,
                     const float *sw, int gs, w4a8_f16 *y, int64_t M, int64_t N, int64_t K,
                     w4a8_stream_t stream)
{
    if (M >= 1 && M <= kMaxMFew && M * K <= kMaxFewCodes) {
        if (N == 0)
            return ok();
        w4a8_status_t st = check_device();
        if (st != W4A8_OK)
            return st;
        launch_few_w4(xq, xs, w4, sw, gs, y, (int)M, (int)N, (int)K, (hipStream_t)stream);
        return check_launch(fn);
    }
    return run_gemm(fn, GemmMode::W4, make_args(xq, xs, w4, sw, y, M, N, K, gs), stream);
}

w4a8_status_t run_quant(const char *fn, const uint16_t *x, int64_t rows, int64_t K, int gs,
                        float qmax, void *q, float *scale, bool int4, w4a8_stream_t stream)
{
    if (rows == 0)
        return ok();
    w4a8_status_t st = check_device();
    if (st != W4A8_OK)
        return st;
    launch_quantize_rows(x, rows, (int)K, gs, qmax, q, scale, int4, (hipStream_t)stream);
    return check_launch(fn);
}

}  // namespace

namespace {

// linear()'s argument rules (no HIP calls): the mode, then the GEMM's rules,
// whatever M is.  Sets *empty for a call with nothing to do.
w4a8_status_t check_linear(const char *fn, w4a8_mode_t mode, const w4a8_f16 *x, int64_t M,
                           int64_t K, const void *w, const float *w_scale, int32_t group_size,
                           int64_t N, w4a8_f16 *y, bool *empty)
{
    *empty = false;
    if (mode == W4A8_MODE_F8) {
        w4a8_status_t st = check_f8(fn, x, nullptr, false, w, w_scale, nullptr, nullptr, false, M, N, K);
        if (st != W4A8_OK)
            return st;
        *empty = M == 0 || N == 0;
        if (!*empty && (!y || !aligned16(y)))
            return fail(y ? W4A8_ERR_ALIGNMENT : W4A8_ERR_INVALID_ARG, "%s: bad y", fn);
        return W4A8_OK;
    }
    if (mode != W4A8_MODE_W8A8_PC && mode != W4A8_MODE_W8A8_PG && mode != W4A8_MODE_W4A8)
        return fail(W4A8_ERR_INVALID_ARG, "%s: unknown mode %d", fn, (int)mode);
    const bool pg = mode != W4A8_MODE_W8A8_PC;
    const int32_t gs = pg ? group_size : 0;
    w4a8_status_t st = check_gemm(fn, x, w, y, w_scale, w_scale, M, N, K, gs, pg, true);
    if (st != W4A8_OK)
        return st;
    if (M == 0 || N == 0) {
        *empty = true;
        return W4A8_OK;
    }
    if (!x || !aligned16(x))
        return fail(x ? W4A8_ERR_ALIGNMENT : W4A8_ERR_INVALID_ARG, "%s: bad x", fn);
    return W4A8_OK;
}

// The layer on checked arguments (check_linear) with the given workspace,
// which may be the static scratch (linear_noalloc).
w4a8_status_t linear_run(const char *fn, w4a8_mode_t mode, const w4a8_f16 *x, int64_t M,
                         int64_t K, const void *w, const float *w_scale, int32_t group_size,
                         int64_t N, w4a8_f16 *y, void *workspace, size_t workspace_bytes,
                         w4a8_stream_t stream)
{
    const int32_t act_gs = (mode == W4A8_MODE_W8A8_PG) ? group_size : 0;
    w4a8_status_t st;
    if (mode == W4A8_MODE_F8) {
        const F8Linear ws(M, K, N);
        st = check_workspace(fn, ws.bytes(), workspace, workspace_bytes);
        if (st != W4A8_OK)
            return st;
        uint8_t *xq = static_cast<uint8_t *>(workspace);
        float *xs = reinterpret_cast<float *>(xq + ws.codes);
        st = quantize_act_f8(x, M, K, xq, xs, stream);
        if (st != W4A8_OK)
            return st;
        F8Args a = make_f8(xq, xs, static_cast<const uint8_t *>(w), w_scale, nullptr, nullptr, M, N, K);
        a.y = y;
        return run_f8(fn, a, false, xq + ws.codes + ws.scales, stream);
    }
    if (M == 1 && K <= kMaxKMv) {                 // decode: the matrix-vector kernels
        switch (mode) {
        case W4A8_MODE_W8A8_PC:
            return int8_mv(x, static_cast<const int8_t *>(w), w_scale, y, N, K, nullptr, nullptr,
                           stream);
        case W4A8_MODE_W8A8_PG:
            return w8a8_mv_pg(x, static_cast<const int8_t *>(w), w_scale, group_size, y, N, K,
                              stream);
        default:
            return w4a8_mv(x, static_cast<const uint8_t *>(w), w_scale, group_size, y, N, K,
                           stream);
        }
    }
    const size_t need = linear_workspace_size(mode, M, K, group_size);
    if (!workspace || workspace_bytes < need ||
        (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
        return fail(W4A8_ERR_WORKSPACE, "%s: workspace of %zu bytes (256-byte aligned) needed, "
                    "got %zu", fn, need, workspace_bytes);
    int8_t *xq = static_cast<int8_t *>(workspace);
    float *xs = reinterpret_cast<float *>(static_cast<char *>(workspace) + align256((size_t)M * K));
    st = quantize_act(x, M, K, act_gs, xq, xs, stream);
    if (st != W4A8_OK)
        return st;
    switch (mode) {
    case W4A8_MODE_W8A8_PC:
        return run_pc(fn, xq, xs, static_cast<const int8_t *>(w), w_scale, y, M, N, K, stream);
    case W4A8_MODE_W8A8_PG:
        return run_gemm(fn, GemmMode::PG,
                        make_args(xq, xs, w, w_scale, y, M, N, K, group_size), stream);
    default:
        return run_w4(fn, xq, xs, static_cast<const uint8_t *>(w), w_scale, group_size, y, M,
                      N, K, stream);
    }
}

// ---- the attention block

bool stride_ok(int64_t stride, int64_t row) { return stride >= row && stride % 8 == 0 && stride <= (int64_t(1) << 40); }

w4a8_status_t check_rotary(const char *fn, const void *x, int64_t x_stride, const int64_t *positions,
                           const float *inv_freq, int64_t T, int32_t heads, int32_t head_dim,
                           int32_t rotary_dim, int32_t axes, const int32_t *sections,
                           const void *out, int64_t out_stride)
{
    if (T < 0 || T > kMaxDim || heads < 0 || heads > 65535)
        return fail(W4A8_ERR_INVALID_ARG, "%s: sizes out of range (T=%lld heads=%d)", fn,
                    (long long)T, (int)heads);
    if (head_dim <= 0 || head_dim % 8 != 0 || head_dim > 1024)
        return fail(W4A8_ERR_SHAPE, "%s: head_dim=%d must be a multiple of 8 in [8, 1024]", fn,
                    (int)head_dim);
    if (rotary_dim <= 0 || rotary_dim % 16 != 0 || rotary_dim > head_dim)
        return fail(W4A8_ERR_SHAPE, "%s: rotary_dim=%d must be a positive multiple of 16 up to "
                    "head_dim=%d", fn, (int)rotary_dim, (int)head_dim);
    if (axes < 1 || axes > 3)
        return fail(W4A8_ERR_SHAPE, "%s: axes=%d must be 1, 2 or 3", fn, (int)axes);
    if (!sections)
        return fail(W4A8_ERR_INVALID_ARG, "%s: null sections", fn);
    int64_t sum = 0;
    for (int a = 0; a < axes; ++a) {
        if (sections[a] < 0)
            return fail(W4A8_ERR_SHAPE, "%s: sections[%d]=%d is negative", fn, a, (int)sections[a]);
        sum += sections[a];
    }
    if (sum != rotary_dim / 2)
        return fail(W4A8_ERR_SHAPE, "%s: the sections sum to %lld, not to rotary_dim / 2 = %d", fn,
                    (long long)sum, (int)(rotary_dim / 2));
    if (T == 0 || heads == 0)
        return W4A8_OK;
    if (!x || !positions || !inv_freq || !out)
        return fail(W4A8_ERR_INVALID_ARG, "%s: null pointer", fn);
    const int64_t row = (int64_t)heads * head_dim;
    if (!stride_ok(x_stride, row) || !stride_ok(out_stride, row))
        return fail(W4A8_ERR_SHAPE, "%s: token strides must be multiples of 8, at least %lld", fn,
                    (long long)row);
    if (x == out && x_stride != out_stride)
        return fail(W4A8_ERR_INVALID_ARG, "%s: in place, the strides must be equal", fn);
    if (!aligned16(x) || !aligned16(out) || !aligned8(positions) || !aligned4(inv_freq))
        return fail(W4A8_ERR_ALIGNMENT, "%s: misaligned tensor", fn);
    return W4A8_OK;
}

// The cache's geometry and buffers.
w4a8_status_t check_cache(const char *fn, const kv4_cache_t *c)
{
    if (!c)
        return fail(W4A8_ERR_INVALID_ARG, "%s: null cache", fn);
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256)
        return fail(W4A8_ERR_SHAPE, "%s: head_dim=%d must be 64, 128 or 256", fn, (int)c->head_dim);
    const int g = c->group_size;
    if ((g != 32 && g != 64 && g != 128 && g != 256) || g > c->head_dim || c->head_dim > 4 * g)
        return fail(W4A8_ERR_SHAPE, "%s: group_size=%d must be 32, 64, 128 or 256, at most "
                    "head_dim=%d and at least a quarter of it", fn, g, (int)c->head_dim);
    const int p = c->page_size;
    if (p < 16 || p > (1 << 20) || (p & (p - 1)) != 0)
        return fail(W4A8_ERR_SHAPE, "%s: page_size=%d must be a power of two in [16, 2^20]", fn, p);
    if (c->kv_heads < 1 || c->kv_heads > 65535)
        return fail(W4A8_ERR_SHAPE, "%s: kv_heads=%d out of range", fn, (int)c->kv_heads);
    if (c->pages < 1 || c->pages > kMaxDim)
        return fail(W4A8_ERR_INVALID_ARG, "%s: pages=%lld out of range", fn, (long long)c->pages);
    if (!c->k || !c->v || !c->k_scale || !c->v_scale)
        return fail(W4A8_ERR_INVALID_ARG, "%s: null cache buffer", fn);
    if (!aligned16(c->k) || !aligned16(c->v) || !aligned16(c->k_scale) || !aligned16(c->v_scale))
        return fail(W4A8_ERR_ALIGNMENT, "%s: cache buffers must be 16-byte aligned", fn);
    return W4A8_OK;
}

Kv4Cache make_cache(const kv4_cache_t *c)
{
    Kv4Cache r;
    r.k = c->k; r.v = c->v; r.ks = c->k_scale; r.vs = c->v_scale;
    r.pages = c->pages;
    r.heads = c->kv_heads; r.shift = __builtin_ctz((unsigned)c->page_size);
    r.D = c->head_dim; r.G = c->group_size;
    return r;
}

// T tokens of a cache: four lanes a row, numbered in 32 bits.
w4a8_status_t check_tokens(const char *fn, int64_t T, const kv4_cache_t *c)
{
    if (T < 0 || T > kMaxDim || T * c->kv_heads > (1 << 29))
        return fail(W4A8_ERR_INVALID_ARG, "%s: T=%lld out of range", fn, (long long)T);
    return W4A8_OK;
}

}  // namespace

extern "C" {

int w4a8_is_available(void) { return check_device() == W4A8_OK ? 1 : 0; }

const char *w4a8_status_string(w4a8_status_t s)
{
    switch (s) {
    case W4A8_OK: return "ok";
    case W4A8_ERR_INVALID_ARG: return "invalid argument";
    case W4A8_ERR_SHAPE: return "unsupported shape";
    case W4A8_ERR_ALIGNMENT: return "misaligned tensor";
    case W4A8_ERR_DEVICE: return "no gfx950 device";
    case W4A8_ERR_LAUNCH: return "kernel launch failed";
    case W4A8_ERR_WORKSPACE: return "workspace too small";
    }
    return "unknown status";
}

const char *w4a8_last_error(void) { return g_err; }

w4a8_status_t quantize_act(const w4a8_f16 *x, int64_t M, int64_t K, int32_t group_size,
                           int8_t *xq, float *x_scale, w4a8_stream_t stream)
{
    w4a8_status_t st = check_quant("quantize_act", x, M, K, group_size, xq, x_scale, false);
    if (st != W4A8_OK)
        return st;
    return run_quant("quantize_act", x, M, K, group_size, 127.0f, xq, x_scale, false, stream);
}

w4a8_status_t quantize_weight_int8(const w4a8_f16 *w, int64_t N, int64_t K, int32_t group_size,
                                   int8_t *wq, float *w_scale, w4a8_stream_t stream)
{
    w4a8_status_t st = check_quant("quantize_weight_int8", w, N, K, group_size, wq, w_scale, false);
    if (st != W4A8_OK)
        return st;
    return run_quant("quantize_weight_int8", w, N, K, group_size, 127.0f, wq, w_scale, false,
                     stream);
}

w4a8_status_t pack_weight_int4(const w4a8_f16 *w, int64_t N, int64_t K, int32_t group_size,
                               uint8_t *w4, float *w_scale, w4a8_stream_t stream)
{
    w4a8_status_t st = check_quant("pack_weight_int4", w, N, K, group_size, w4, w_scale, true);
    if (st != W4A8_OK)
        return st;
    return run_quant("pack_weight_int4", w, N, K, group_size, 7.0f, w4, w_scale, true, stream);
}

w4a8_status_t w8a8_gemm_pc(const int8_t *xq, const float *x_scale, const int8_t *wq,
                           const float *w_scale, w4a8_f16 *y, int64_t M, int64_t N, int64_t K,
                           w4a8_stream_t stream)
{
    w4a8_status_t st = check_gemm("w8a8_gemm_pc", xq, wq, y, x_scale, w_scale, M, N, K, 0, false,
                                  true);
    if (st != W4A8_OK)
        return st;
    return run_pc("w8a8_gemm_pc", xq, x_scale, wq, w_scale, y, M, N, K, stream);
}

w4a8_status_t w8a8_gemm_pg(const int8_t *xq, const float *x_scale, const int8_t *wq,
                           const float *w_scale, int32_t group_size, w4a8_f16 *y, int64_t M,
                           int64_t N, int64_t K, w4a8_stream_t stream)
{
    w4a8_status_t st = check_gemm("w8a8_gemm_pg", xq, wq, y, x_scale, w_scale, M, N, K, group_size,
                                  true, true);
    if (st != W4A8_OK)
        return st;
    return run_gemm("w8a8_gemm_pg", GemmMode::PG,
                    make_args(xq, x_scale, wq, w_scale, y, M, N, K, group_size), stream);
}

w4a8_status_t w4a8_gemm(const int8_t *xq, const float *x_scale, const uint8_t *w4,
                        const float *w_scale, int32_t group_size, w4a8_f16 *y, int64_t M,
                        int64_t N, int64_t K, w4a8_stream_t stream)
{
    w4a8_status_t st = check_gemm("w4a8_gemm", xq, w4, y, x_scale, w_scale, M, N, K, group_size,
                                  true, true);
    if (st != W4A8_OK)
        return st;
    return run_w4("w4a8_gemm", xq, x_scale, w4, w_scale, group_size, y, M, N, K, stream);
}

w4a8_status_t int8_mv(const w4a8_f16 *x, const int8_t *wq, const float *w_scale, w4a8_f16 *y,
                      int64_t N, int64_t K, int8_t *xq_out, float *x_scale_out,
                      w4a8_stream_t stream)
{
    w4a8_status_t st = check_mv(x, wq, w_scale, y, N, K, xq_out, x_scale_out);
    if (st != W4A8_OK)
        return st;
    if (N == 0 && !xq_out && !x_scale_out)
        return ok();
    st = check_device();
    if (st != W4A8_OK)
        return st;
    if (N == 0) {
        // nothing to multiply, but the caller asked for the token's codes:
        // the codes come from the activation quantizer (same rule)
        if (!xq_out || !x_scale_out)
            return fail(W4A8_ERR_INVALID_ARG, "int8_mv: N == 0 needs both or neither export");
        launch_quantize_rows(x, 1, (int)K, 0, 127.0f, xq_out, x_scale_out, false,
                             (hipStream_t)stream);
        return check_launch("int8_mv");
    }
    launch_int8_mv(x, wq, w_scale, y, (int)N, (int)K, xq_out, x_scale_out, (hipStream_t)stream);
    return check_launch("int8_mv");
}

w4a8_status_t w8a8_mv_pg(const w4a8_f16 *x, const int8_t *wq, const float *w_scale,
                         int32_t group_size, w4a8_f16 *y, int64_t N, int64_t K,
                         w4a8_stream_t stream)
{
    w4a8_status_t st = check_mv_group("w8a8_mv_pg", x, wq, w_scale, y, N, K, group_size);
    if (st != W4A8_OK)
        return st;
    if (N == 0)
        return ok();
    int cu = 0;
    st = check_device(&cu);
    if (st != W4A8_OK)
        return st;
    launch_mv_group(false, group_size, x, reinterpret_cast<const uint8_t *>(wq), w_scale, y,
                    (int)N, (int)K, cu, (hipStream_t)stream);
    return check_launch("w8a8_mv_pg");
}

w4a8_status_t w4a8_mv(const w4a8_f16 *x, const uint8_t *w4, const float *w_scale,
                      int32_t group_size, w4a8_f16 *y, int64_t N, int64_t K,
                      w4a8_stream_t stream)
{
    w4a8_status_t st = check_mv_group("w4a8_mv", x, w4, w_scale, y, N, K, group_size);
    if (st != W4A8_OK)
        return st;
    if (N == 0)
        return ok();
    int cu = 0;
    st = check_device(&cu);
    if (st != W4A8_OK)
        return st;
    launch_mv_group(true, group_size, x, w4, w_scale, y, (int)N, (int)K, cu, (hipStream_t)stream);
    return check_launch("w4a8_mv");
}

size_t linear_workspace_size(w4a8_mode_t mode, int64_t M, int64_t K, int32_t group_size)
{
    if (M <= 0 || K <= 0)
        return 0;
    if (mode == W4A8_MODE_F8)
        return F8Linear(M, K).bytes();
    if (M == 1 && K <= kMaxKMv)                   // the matrix-vector kernels need none
        return 0;
    int64_t groups = 1;
    if (mode == W4A8_MODE_W8A8_PG && group_size > 0)
        groups = K / group_size;
    return align256((size_t)M * (size_t)K) + align256((size_t)M * (size_t)groups * sizeof(float));
}

w4a8_status_t linear(w4a8_mode_t mode, const w4a8_f16 *x, int64_t M, int64_t K, const void *w,
                     const float *w_scale, int32_t group_size, int64_t N, w4a8_f16 *y,
                     void *workspace, size_t workspace_bytes, w4a8_stream_t stream)
{
    bool empty;
    w4a8_status_t st = check_linear("linear", mode, x, M, K, w, w_scale, group_size, N, y, &empty);
    if (st != W4A8_OK || empty)
        return st == W4A8_OK ? ok() : st;
    return linear_run("linear", mode, x, M, K, w, w_scale, group_size, N, y, workspace,
                      workspace_bytes, stream);
}

w4a8_status_t linear_noalloc(w4a8_mode_t mode, const w4a8_f16 *x, int64_t M, int64_t K,
                             const void *w, const float *w_scale, int32_t group_size, int64_t N,
                             w4a8_f16 *y, w4a8_stream_t stream)
{
    const char *fn = "linear_noalloc";
    bool empty;
    w4a8_status_t st = check_linear(fn, mode, x, M, K, w, w_scale, group_size, N, y, &empty);
    if (st != W4A8_OK || empty)
        return st == W4A8_OK ? ok() : st;
    const size_t need = mode == W4A8_MODE_F8 ? F8Linear(M, K, N).bytes()
                                             : linear_workspace_size(mode, M, K, group_size);
    if (need > kScratchBytes)
        return fail(W4A8_ERR_WORKSPACE, "%s: M=%lld, K=%lld need %zu bytes of scratch; the "
                    "static array holds %zu (call linear() with a workspace)", fn, (long long)M,
                    (long long)K, need, kScratchBytes);
    void *ws = nullptr;
    if (need > 0) {
        st = check_device();
        if (st != W4A8_OK)
            return st;
        st = scratch_address(&ws);
        if (st != W4A8_OK)
            return st;
    }
    return linear_run(fn, mode, x, M, K, w, w_scale, group_size, N, y, ws, kScratchBytes, stream);
}

w4a8_status_t w8a8_gemm_i32(const int8_t *xq, const int8_t *wq, int32_t *c, int64_t M, int64_t N,
                            int64_t K, w4a8_stream_t stream)
{
    w4a8_status_t st = check_gemm("w8a8_gemm_i32", xq, wq, c, nullptr, nullptr, M, N, K, 0, false,
                                  false);
    if (st != W4A8_OK)
        return st;
    return run_gemm("w8a8_gemm_i32", GemmMode::I32,
                    make_args(xq, nullptr, wq, nullptr, c, M, N, K, 0), stream);
}

w4a8_status_t w8a8_gemm_pg_partials(const int8_t *xq, const int8_t *wq, int32_t group_size,
                                    int32_t *p, int64_t M, int64_t N, int64_t K,
                                    w4a8_stream_t stream)
{
    w4a8_status_t st = check_gemm("w8a8_gemm_pg_partials", xq, wq, p, nullptr, nullptr, M, N, K,
                                  group_size, true, false);
    if (st != W4A8_OK)
        return st;
    return run_gemm("w8a8_gemm_pg_partials", GemmMode::PG_PARTIALS,
                    make_args(xq, nullptr, wq, nullptr, p, M, N, K, group_size), stream);
}

w4a8_status_t w4a8_gemm_partials(const int8_t *xq, const uint8_t *w4, int32_t group_size,
                                 int32_t *p, int64_t M, int64_t N, int64_t K,
                                 w4a8_stream_t stream)
{
    w4a8_status_t st = check_gemm("w4a8_gemm_partials", xq, w4, p, nullptr, nullptr, M, N, K,
                                  group_size, true, false);
    if (st != W4A8_OK)
        return st;
    return run_gemm("w4a8_gemm_partials", GemmMode::W4_PARTIALS,
                    make_args(xq, nullptr, w4, nullptr, p, M, N, K, group_size), stream);
}

w4a8_status_t w8a16_gemm(const w4a8_f16 *x, const int8_t *wq, const float *w_scale, w4a8_f16 *y,
                         int64_t M, int64_t N, int64_t K, w4a8_stream_t stream)
{
    const char *fn = "w8a16_gemm";
    if (M < 0 || N < 0 || K < 0 || M > kMaxDim || N > kMaxDim || K > kMaxDim)
        return fail(W4A8_ERR_INVALID_ARG, "%s: sizes out of range (M=%lld N=%lld K=%lld)", fn,
                    (long long)M, (long long)N, (long long)K);
    if (K == 0 || K % 64 != 0)
        return fail(W4A8_ERR_SHAPE, "%s: K=%lld must be a positive multiple of 64", fn,
                    (long long)K);
    if ((M + 127) / 128 > 65535)
        return fail(W4A8_ERR_SHAPE, "%s: M=%lld exceeds 65535 * 128 rows", fn, (long long)M);
    if (M == 0 || N == 0)
        return ok();
    if (!x || !wq || !w_scale || !y)
        return fail(W4A8_ERR_INVALID_ARG, "%s: null pointer", fn);
    if (!aligned16(x) || !aligned16(wq) || !aligned16(y) || !aligned4(w_scale))
        return fail(W4A8_ERR_ALIGNMENT, "%s: tensors must be 16-byte aligned", fn);
    w4a8_status_t st = check_device();
    if (st != W4A8_OK)
        return st;
    if (M == 1 && K <= kMaxKWoMv)                     // one token: the matrix-vector form
        launch_wo_mv(false, reinterpret_cast<const uint16_t *>(x), wq, w_scale, 0,
                     reinterpret_cast<uint16_t *>(y), (int)N, (int)K, (hipStream_t)stream);
    else
        launch_w8a16(reinterpret_cast<const uint16_t *>(x), wq, w_scale,
                     reinterpret_cast<uint16_t *>(y), (int)M, (int)N, (int)K, (hipStream_t)stream);
    return check_launch(fn);
}

w4a8_status_t w4a16_gemm(const w4a8_f16 *x, const uint8_t *w4, const float *w_scale,
                         int32_t group_size, w4a8_f16 *y, int64_t M, int64_t N, int64_t K,
                         w4a8_stream_t stream)
{
    const char *fn = "w4a16_gemm";
    if (M < 0 || N < 0 || K < 0 || M > kMaxDim || N > kMaxDim || K > kMaxDim)
        return fail(W4A8_ERR_INVALID_ARG, "%s: sizes out of range (M=%lld N=%lld K=%lld)", fn,
                    (long long)M, (long long)N, (long long)K);
    if (!(group_size == 64 || group_size == 128))
        return fail(W4A8_ERR_SHAPE, "%s: group_size=%d must be 64 or 128", fn, (int)group_size);
    if (K == 0 || K % 64 != 0 || K % group_size != 0)
        return fail(W4A8_ERR_SHAPE, "%s: K=%lld must be a positive multiple of 64 and of "
                    "group_size", fn, (long long)K);
    if ((M + 127) / 128 > 65535)
        return fail(W4A8_ERR_SHAPE, "%s: M=%lld exceeds 65535 * 128 rows", fn, (long long)M);
    if (M == 0 || N == 0)
        return ok();
    if (!x || !w4 || !w_scale || !y)
        return fail(W4A8_ERR_INVALID_ARG, "%s: null pointer", fn);
    if (!aligned16(x) || !aligned16(w4) || !aligned16(y) || !aligned4(w_scale))
        return fail(W4A8_ERR_ALIGNMENT, "%s: tensors must be 16-byte aligned", fn);
    w4a8_status_t st = check_device();
    if (st != W4A8_OK)
        return st;
    if (M == 1 && K <= kMaxKWoMv)                     // one token: the matrix-vector form
        launch_wo_mv(true, reinterpret_cast<const uint16_t *>(x), w4, w_scale, (int)group_size,
                     reinterpret_cast<uint16_t *>(y), (int)N, (int)K, (hipStream_t)stream);
    else
        launch_w4a16(reinterpret_cast<const uint16_t *>(x), w4, w_scale, (int)group_size,
                     reinterpret_cast<uint16_t *>(y), (int)M, (int)N, (int)K, (hipStream_t)stream);
    return check_launch(fn);
}

w4a8_status_t gemm_tile_config(w4a8_gemm_op_t op, int64_t M, int64_t N, int64_t K,
                               int32_t group_size, int64_t *out)
{
    const char *fn = "gemm_tile_config";
    if (!out)
        return fail(W4A8_ERR_INVALID_ARG, "%s: null out", fn);
    GemmMode mode;
    bool pergroup = true, few = false;
    switch (op) {
    case W4A8_OP_GEMM_PC: mode = GemmMode::PC; pergroup = false; few = true; break;
    case W4A8_OP_GEMM_I32: mode = GemmMode::I32; pergroup = false; break;
    case W4A8_OP_GEMM_PG: mode = GemmMode::PG; break;
    case W4A8_OP_PG_PARTIALS: mode = GemmMode::PG_PARTIALS; break;
    case W4A8_OP_GEMM_W4A8: mode = GemmMode::W4; few = true; break;
    case W4A8_OP_W4A8_PARTIALS: mode = GemmMode::W4_PARTIALS; break;
    default: return fail(W4A8_ERR_INVALID_ARG, "%s: unknown op %d", fn, (int)op);
    }
    // the entry point's own shape rules (pointers are not inspected)
    static const int8_t dummy[16] __attribute__((aligned(16))) = {0};
    const float *fs = reinterpret_cast<const float *>(dummy);
    w4a8_status_t st = check_gemm(fn, dummy, dummy, dummy, fs, fs, M, N, K,
                                  pergroup ? group_size : 0, pergroup, false);
    if (st != W4A8_OK)
        return st;
    for (int i = 0; i < 6; ++i)
        out[i] = 0;
    if (M == 0 || N == 0)
        return ok();
    int num_cu = 0;
    st = check_device(&num_cu);
    if (st != W4A8_OK)
        return st;
    if (few && M >= 1 && M <= kMaxMFew && M * K <= kMaxFewCodes)
        return ok();                              // the few-token matrix-vector form
    GemmArgs a = make_args(nullptr, nullptr, nullptr, nullptr, nullptr, M, N, K,
                           pergroup ? group_size : 0);
    a.num_cu = num_cu;
    const TileInfo t = gemm_info(mode, a);
    out[0] = t.bm;
    out[1] = t.bn;
    out[2] = t.waves;
    out[3] = t.grid;
    out[4] = t.tiles;
    out[5] = t.per_cu;
    return ok();
}

w4a8_status_t rotary_axes(const w4a8_f16 *x, int64_t x_stride, const int64_t *positions,
                          const float *inv_freq, int64_t T, int32_t heads, int32_t head_dim,
                          int32_t rotary_dim, int32_t axes, const int32_t *sections,
                          int32_t interleaved, w4a8_f16 *out, int64_t out_stride,
                          w4a8_stream_t stream)
{
    const char *fn = "rotary_axes";
    w4a8_status_t st = check_rotary(fn, x, x_stride, positions, inv_freq, T, heads, head_dim,
                                    rotary_dim, axes, sections, out, out_stride);
    if (st != W4A8_OK)
        return st;
    if (T == 0 || heads == 0)
        return ok();
    st = check_device();
    if (st != W4A8_OK)
        return st;
    launch_rotary(x, x_stride, positions, inv_freq, T, heads, head_dim, rotary_dim, axes, sections,
                  interleaved != 0, out, out_stride, (hipStream_t)stream);
    return check_launch(fn);
}

w4a8_status_t kv4_write(const w4a8_f16 *k, int64_t k_stride, const w4a8_f16 *v, int64_t v_stride,
                        const int64_t *slots, int64_t T, const kv4_cache_t *cache,
                        w4a8_stream_t stream)
{
    const char *fn = "kv4_write";
    w4a8_status_t st = check_cache(fn, cache);
    if (st == W4A8_OK)
        st = check_tokens(fn, T, cache);
    if (st != W4A8_OK)
        return st;
    if (T == 0)
        return ok();
    if (!k || !v || !slots)
        return fail(W4A8_ERR_INVALID_ARG, "%s: null pointer", fn);
    const int64_t row = (int64_t)cache->kv_heads * cache->head_dim;
    if (!stride_ok(k_stride, row) || !stride_ok(v_stride, row))
        return fail(W4A8_ERR_SHAPE, "%s: token strides must be multiples of 8, at least %lld", fn,
                    (long long)row);
    if (!aligned16(k) || !aligned16(v) || !aligned8(slots))
        return fail(W4A8_ERR_ALIGNMENT, "%s: misaligned tensor", fn);
    st = check_device();
    if (st != W4A8_OK)
        return st;
    launch_kv4_write(k, k_stride, v, v_stride, slots, T, make_cache(cache), (hipStream_t)stream);
    return check_launch(fn);
}

w4a8_status_t kv4_read(const kv4_cache_t *cache, const int64_t *slots, int64_t T, w4a8_f16 *k,
                       w4a8_f16 *v, w4a8_stream_t stream)
{
    const char *fn = "kv4_read";
    w4a8_status_t st = check_cache(fn, cache);
    if (st == W4A8_OK)
        st = check_tokens(fn, T, cache);
    if (st != W4A8_OK)
        return st;
    if (T == 0)
        return ok();
    if (!k || !v || !slots)
        return fail(W4A8_ERR_INVALID_ARG, "%s: null pointer", fn);
    if (!aligned16(k) || !aligned16(v) || !aligned8(slots))
        return fail(W4A8_ERR_ALIGNMENT, "%s: misaligned tensor", fn);
    st = check_device();
    if (st != W4A8_OK)
        return st;
    launch_kv4_read(make_cache(cache), slots, T, k, v, (hipStream_t)stream);
    return check_launch(fn);
}

w4a8_status_t quantize_act_f8(const w4a8_f16 *x, int64_t M, int64_t K, uint8_t *xq, float *x_scale,
                              w4a8_stream_t stream)
{
    const char *fn = "quantize_act_f8";
    if (M < 0 || K < 0 || M > kMaxRowsF8 || K > kMaxKGemm)
        return fail(W4A8_ERR_INVALID_ARG, "%s: sizes out of range (M=%lld K=%lld)", fn, (long long)M,
                    (long long)K);
    w4a8_status_t st = check_quant(fn, x, M, K, 0, xq, x_scale, false);
    if (st != W4A8_OK)
        return st;
    if (M == 0)
        return ok();
    st = check_device();
    if (st != W4A8_OK)
        return st;
    launch_quantize_act_f8(x, M, (int)K, xq, x_scale, (hipStream_t)stream);
    return check_launch(fn);
}

w4a8_status_t quantize_weight_f8(const w4a8_f16 *w, int64_t N, int64_t K, uint8_t *wq, float *w_scale,
                                 w4a8_stream_t stream)
{
    const char *fn = "quantize_weight_f8";
    if (N < 0 || K < 0 || N > kMaxDim || K > kMaxKGemm)
        return fail(W4A8_ERR_INVALID_ARG, "%s: sizes out of range (N=%lld K=%lld)", fn, (long long)N,
                    (long long)K);
    w4a8_status_t st = check_quant(fn, w, N, K, 0, wq, w_scale, false);
    if (st != W4A8_OK)
        return st;
    if (((N + 127) / 128) * ((K + 127) / 128) >= (1 << 24))
        return fail(W4A8_ERR_SHAPE, "%s: N=%lld x K=%lld has more than 2^24 - 1 blocks", fn, (long long)N,
                    (long long)K);
    if (N == 0)
        return ok();
    st = check_device();
    if (st != W4A8_OK)
        return st;
    launch_quantize_weight_f8(w, N, (int)K, wq, w_scale, (hipStream_t)stream);
    return check_launch(fn);
}

w4a8_status_t rmsnorm_quant(w4a8_mode_t mode, const w4a8_f16 *x, const w4a8_f16 *residual,
                            const w4a8_f16 *gain, float eps, int64_t M, int64_t K, int32_t group_size,
                            void *q, float *scale, w4a8_f16 *residual_out, w4a8_stream_t stream)
{
    const char *fn = "rmsnorm_quant";
    if (mode != W4A8_MODE_W8A8_PC && mode != W4A8_MODE_W8A8_PG && mode != W4A8_MODE_W4A8 &&
        mode != W4A8_MODE_F8)
        return fail(W4A8_ERR_INVALID_ARG, "%s: unknown mode %d", fn, (int)mode);
    if (M < 0 || K < 0 || M > kMaxRowsF8 || K > kMaxKGemm)
        return fail(W4A8_ERR_INVALID_ARG, "%s: sizes out of range (M=%lld K=%lld)", fn, (long long)M,
                    (long long)K);
    const bool groups = mode == W4A8_MODE_W8A8_PG;
    if (groups && group_size != 64 && group_size != 128)
        return fail(W4A8_ERR_SHAPE, "%s: group_size=%d must be 64 or 128", fn, (int)group_size);
    if (!(eps >= 0.0f) || eps > 0x1p127f)
        return fail(W4A8_ERR_INVALID_ARG, "%s: eps must be finite and not negative", fn);
    w4a8_status_t st = check_quant(fn, x, M, K, groups ? group_size : 0, q, scale, false);
    if (st != W4A8_OK)
        return st;
    if (M == 0)
        return ok();
    if (!gain)
        return fail(W4A8_ERR_INVALID_ARG, "%s: null gain", fn);
    if (!aligned16(gain) || !aligned16(residual) || !aligned16(residual_out))
        return fail(W4A8_ERR_ALIGNMENT, "%s: tensors must be 16-byte aligned", fn);
    st = check_device();
    if (st != W4A8_OK)
        return st;
    NormArgs a;
    a.x = x; a.residual = residual; a.gain = gain; a.sum = residual_out;
    a.q = static_cast<uint8_t *>(q); a.scale = scale;
    a.M = M; a.K = (int)K; a.eps = eps;
    const NormOut out = mode == W4A8_MODE_F8 ? NormOut::F8
                        : !groups            ? NormOut::INT8_ROW
                        : group_size == 64   ? NormOut::INT8_64
                                             : NormOut::INT8_128;
    launch_rmsnorm_quant(out, a, (hipStream_t)stream);
    return check_launch(fn);
}

size_t f8_gemm_workspace_size(int64_t M, int64_t N, int64_t K)
{
    return f8_workspace(M, N, K, false, false);
}

w4a8_status_t f8_gemm(const uint8_t *xq, const float *x_scale, const uint8_t *wq, const float *w_scale,
                      w4a8_f16 *y, int64_t M, int64_t N, int64_t K, void *workspace,
                      size_t workspace_bytes, w4a8_stream_t stream)
{
    const char *fn = "f8_gemm";
    w4a8_status_t st = check_f8(fn, xq, x_scale, true, wq, w_scale, nullptr, nullptr, false, M, N, K);
    if (st != W4A8_OK)
        return st;
    if (M == 0 || N == 0)
        return ok();
    if (!y || !aligned16(y))
        return fail(y ? W4A8_ERR_ALIGNMENT : W4A8_ERR_INVALID_ARG, "%s: bad y", fn);
    st = check_workspace(fn, f8_gemm_workspace_size(M, N, K), workspace, workspace_bytes);
    if (st != W4A8_OK)
        return st;
    F8Args a = make_f8(xq, x_scale, wq, w_scale, nullptr, nullptr, M, N, K);
    a.y = y;
    return run_f8(fn, a, false, workspace, stream);
}

size_t f8_gemm_gated_workspace_size(int64_t M, int64_t N, int64_t K, int32_t quantize)
{
    return f8_workspace(M, N, K, true, quantize != 0);
}

w4a8_status_t f8_gemm_gated(const uint8_t *xq, const float *x_scale, const uint8_t *w_gate,
                            const float *gate_scale, const uint8_t *w_up, const float *up_scale,
                            w4a8_activation_t activation, int64_t M, int64_t N, int64_t K, w4a8_f16 *y,
                            uint8_t *yq, float *y_scale, void *workspace, size_t workspace_bytes,
                            w4a8_stream_t stream)
{
    const char *fn = "f8_gemm_gated";
    w4a8_status_t st = check_f8(fn, xq, x_scale, true, w_gate, gate_scale, w_up, up_scale, true, M, N, K);
    if (st != W4A8_OK)
        return st;
    if (activation != W4A8_ACT_SILU && activation != W4A8_ACT_GELU_TANH)
        return fail(W4A8_ERR_INVALID_ARG, "%s: unknown activation %d", fn, (int)activation);
    if (M == 0 || N == 0)
        return ok();
    if (y ? (yq || y_scale) : (!yq || !y_scale))
        return fail(W4A8_ERR_INVALID_ARG, "%s: either y, or yq and y_scale", fn);
    if (!aligned16(y) || !aligned16(yq) || !aligned4(y_scale))
        return fail(W4A8_ERR_ALIGNMENT, "%s: tensors must be 16-byte aligned", fn);
    st = check_workspace(fn, f8_gemm_gated_workspace_size(M, N, K, y ? 0 : 1), workspace, workspace_bytes);
    if (st != W4A8_OK)
        return st;
    F8Args a = make_f8(xq, x_scale, w_gate, gate_scale, w_up, up_scale, M, N, K);
    a.y = y; a.yq = yq; a.ys = y_scale;
    a.gelu = activation == W4A8_ACT_GELU_TANH;
    return run_f8(fn, a, true, workspace, stream);
}

size_t kv4_attention_workspace_size(int32_t q_heads, int32_t kv_heads, int32_t head_dim, int64_t T,
                                    int64_t sequences, int32_t max_q)
{
    if (q_heads <= 0 || kv_heads <= 0 || q_heads % kv_heads != 0 || head_dim <= 0 || T <= 0 ||
        sequences <= 0 || sequences > (1 << 20) || max_q <= 0)
        return 0;
    return kv4_attention_workspace(q_heads, kv_heads, head_dim, T, (int)sequences, max_q);
}

w4a8_status_t kv4_attention(const w4a8_f16 *q, int64_t q_stride, int64_t T, int32_t q_heads,
                            const kv4_cache_t *cache, const int32_t *page_table,
                            int32_t max_pages, const int32_t *kv_lens, const int32_t *q_starts,
                            int64_t sequences, int32_t max_q, int32_t causal, int32_t window,
                            float scale, w4a8_f16 *out, float *lse, void *workspace,
                            size_t workspace_bytes, w4a8_stream_t stream)
{
    const char *fn = "kv4_attention";
    w4a8_status_t st = check_cache(fn, cache);
    if (st != W4A8_OK)
        return st;
    if (T < 0 || sequences < 0 || T > kMaxDim || sequences > (1 << 20) || max_q < 0 ||
        q_heads < 1 || q_heads > 65535 || T * q_heads > kMaxDim ||
        sequences * cache->kv_heads > (1 << 28) || max_pages < 0)
        return fail(W4A8_ERR_INVALID_ARG, "%s: sizes out of range (T=%lld q_heads=%d sequences=%lld "
                    "max_q=%d max_pages=%d)", fn, (long long)T, (int)q_heads, (long long)sequences,
                    (int)max_q, (int)max_pages);
    if (q_heads % cache->kv_heads != 0)
        return fail(W4A8_ERR_SHAPE, "%s: q_heads=%d is not a multiple of kv_heads=%d", fn,
                    (int)q_heads, (int)cache->kv_heads);
    const int64_t most = (int64_t)max_pages * cache->page_size;
    if (most > (int64_t(1) << 30) || (most / 32 + 1) * sequences * cache->kv_heads > (int64_t(1) << 45))
        return fail(W4A8_ERR_SHAPE, "%s: max_pages=%d pages of %d tokens are too many (2^30 a "
                    "sequence, 2^50 in all)", fn, (int)max_pages, (int)cache->page_size);
    if (window < 0 || (window > 0 && !causal))
        return fail(W4A8_ERR_INVALID_ARG, "%s: window=%d needs causal and must not be negative", fn,
                    (int)window);
    if (!(scale > 0.0f) || scale > 0x1p127f)             // scale * log2(e) has to be finite
        return fail(W4A8_ERR_INVALID_ARG, "%s: scale must be positive and at most 2^127", fn);
    if (!q_starts && (T != sequences || (T > 0 && max_q < 1)))
        return fail(W4A8_ERR_SHAPE, "%s: without q_starts, T=%lld must equal sequences=%lld and "
                    "max_q be at least 1", fn, (long long)T, (long long)sequences);
    if (T == 0 || sequences == 0 || max_q == 0)
        return T == 0 ? ok() : fail(W4A8_ERR_SHAPE, "%s: %lld query rows in no sequence", fn,
                                    (long long)T);
    if (!q || !kv_lens || !out || (max_pages > 0 && !page_table))
        return fail(W4A8_ERR_INVALID_ARG, "%s: null pointer", fn);
    if (!stride_ok(q_stride, (int64_t)q_heads * cache->head_dim))
        return fail(W4A8_ERR_SHAPE, "%s: the token stride must be a multiple of 8, at least %lld",
                    fn, (long long)q_heads * cache->head_dim);
    if (!aligned16(q) || !aligned16(out) || !aligned4(page_table) || !aligned4(kv_lens) ||
        !aligned4(q_starts) || !aligned4(lse))
        return fail(W4A8_ERR_ALIGNMENT, "%s: misaligned tensor", fn);
    Kv4AttnArgs a;
    a.q = q; a.q_stride = q_stride; a.T = T; a.q_heads = q_heads;
    a.group = q_heads / cache->kv_heads;
    a.table = page_table; a.max_pages = max_pages; a.kv_lens = kv_lens; a.q_starts = q_starts;
    a.B = (int)sequences;
    a.max_q = (int)(max_q < T ? max_q : T);
    a.causal = causal != 0; a.window = window; a.scale = scale;
    a.out = out; a.lse = lse; a.workspace = workspace; a.tag = next_tag();
    const Kv4Cache kc = make_cache(cache);
    if (!kv4_attention_fits(kc, a))
        return fail(W4A8_ERR_INVALID_ARG, "%s: sequences=%lld with %d kv heads take more workgroups "
                    "than a launch holds", fn, (long long)sequences, (int)cache->kv_heads);
    const size_t need = kv4_attention_workspace_size(q_heads, cache->kv_heads, cache->head_dim, T,
                                                     sequences, max_q);
    if (need > 0 && (!workspace || workspace_bytes < need ||
                     (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0))
        return fail(W4A8_ERR_WORKSPACE, "%s: workspace of %zu bytes (256-byte aligned) needed, got "
                    "%zu", fn, need, workspace_bytes);
    st = check_device();
    if (st != W4A8_OK)
        return st;
    launch_kv4_attention(kc, a, (hipStream_t)stream);
    return check_launch(fn);
}

}  // extern "C"

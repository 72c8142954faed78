// Quantization to e4m3 in blocks of 128 (activations per token, weights in
// 128 x 128 blocks), and the root-mean-square norm with the residual's
// addition whose output is quantized for the linear layer behind it.
#include "f8.hpp"
#include "f8_device.hpp"

namespace w4a8 {

namespace {

// The codes of a 16-byte chunk of fp16 values.
__device__ __forceinline__ uint2 f8_chunk8(uint4 v, float s, float r)
{
    return make_uint2(f8_codes4<false>(lo_h2f(v.x), hi_h2f(v.x), lo_h2f(v.y), hi_h2f(v.y), s, r),
                      f8_codes4<false>(lo_h2f(v.z), hi_h2f(v.z), lo_h2f(v.w), hi_h2f(v.w), s, r));
}

// The largest |x| of fp16 values, as fp16 bits, to fp32 bits: infinities and
// NaN stay above every finite value.
__device__ __forceinline__ uint32_t amax_h2f_bits(uint32_t m) { return __float_as_uint(h2f((uint16_t)m)); }

// A row's wavefronts take its runs of 512 values, one each while a launch can
// number them; 16 lanes own a block of 128, 8 values a lane.  Bound by latency
// where rows are few, by memory where they are many: against one wavefront a
// row 1 x 4096 1.9 us (4.4), 32 x 14336 2.2 (17.8), 517 x 4096 3.3 (7.0), 4516 x
// 4096 14.0 (14.8; 4.0 TB/s), 4516 x 1024 5.4 (5.1).
__global__ __launch_bounds__(256) void quant_act_f8_kernel(const uint16_t *__restrict__ x,
                                                           uint8_t *__restrict__ q,
                                                           float *__restrict__ scale, int64_t rows,
                                                           int K, int waves)
{
    const int lane = threadIdx.x & 63;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(blockIdx.x * 4 + (threadIdx.x >> 6));
    const int64_t row = wave / (uint32_t)waves;
    if (row >= rows)
        return;
    const int first = (int)(wave % (uint32_t)waves);
    const int nch = K >> 3;
    const uint4 *xr = reinterpret_cast<const uint4 *>(x + row * (int64_t)K);
    for (int base = 64 * first; base < nch; base += 64 * waves) {
        const int c = base + lane;
        const bool valid = c < nch;
        const uint4 v = valid ? xr[c] : make_uint4(0u, 0u, 0u, 0u);
        const uint32_t m = group_max_u32<16>(absmax_bits8(v));
        float s, r;
        f8_block_scale<false>(amax_h2f_bits(m), s, r);
        if (!valid)
            continue;
        if ((lane & 15) == 0)
            scale[(int64_t)(c >> 4) * rows + row] = s;
        reinterpret_cast<uint2 *>(q + row * (int64_t)K)[c] = f8_chunk8(v, s, r);
    }
}

// One workgroup a 128 x 128 block, in registers: wave w owns rows 4 w .. 4 w + 3
// of every sixteen, 16 lanes each.  Bound by memory: 12288 x 4096 27.4 us (5.5
// TB/s, part of it from the caches), 4096 x 4096 10.0.
__global__ __launch_bounds__(256) void quant_weight_f8_kernel(const uint16_t *__restrict__ w,
                                                              uint8_t *__restrict__ q,
                                                              float *__restrict__ scale, int64_t N,
                                                              int K, int kblocks)
{
    __shared__ uint32_t top[4];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t nb = blockIdx.x / kblocks;
    const int kb = blockIdx.x % kblocks;
    const int c = kb * 16 + (lane & 15);
    uint4 v[8];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t row = nb * kF8Block + i * 16 + wave * 4 + (lane >> 4);
        const bool valid = row < N && c * 8 < K;
        v[i] = valid ? reinterpret_cast<const uint4 *>(w + row * (int64_t)K)[c] : make_uint4(0u, 0u, 0u, 0u);
        m = max(m, absmax_bits8(v[i]));
    }
    m = group_max_u32<64>(m);
    if (lane == 0)
        top[wave] = m;
    __syncthreads();
    m = max(max(top[0], top[1]), max(top[2], top[3]));
    float s, r;
    f8_block_scale<false>(amax_h2f_bits(m), s, r);
    if (threadIdx.x == 0)
        scale[nb * kblocks + kb] = s;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t row = nb * kF8Block + i * 16 + wave * 4 + (lane >> 4);
        if (row < N && c * 8 < K)
            reinterpret_cast<uint2 *>(q + row * (int64_t)K)[c] = f8_chunk8(v[i], s, r);
    }
}

// ---- rmsnorm_quant

struct Eight {
    float v[8];
};

__device__ __forceinline__ Eight widen(uint4 u)
{
    return {{lo_h2f(u.x), hi_h2f(u.x), lo_h2f(u.y), hi_h2f(u.y), lo_h2f(u.z), hi_h2f(u.z), lo_h2f(u.w),
             hi_h2f(u.w)}};
}

template <typename T> __device__ __forceinline__ T wave_sum(T v)
{
#pragma unroll
    for (int d = 32; d > 0; d >>= 1)
        v += __shfl_xor(v, d);
    return v;
}

// fl32(v / s) to an int8 code (f8_quotient's steps and its domain); v is no more
// than the slice's largest, but the quotient is taken in fp32, so it is clamped
// as the rule says.
__device__ __forceinline__ uint32_t int8_codes4(const float *v, float s, float r)
{
    int c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        c[i] = r == 0.0f ? 0 : quant_code_corrected(v[i], s, r, 127.0f);
    return pack_i8x4(c[0], c[1], c[2], c[3]);
}

// x + residual in fp32.
__device__ __forceinline__ Eight norm_sum(uint4 x, uint4 r)
{
    Eight h = widen(x);
    const Eight t = widen(r);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        h.v[i] += t.v[i];
    return h;
}

__device__ __forceinline__ void norm_squares(const Eight &h, float &ss)
{
#pragma unroll
    for (int i = 0; i < 8; ++i)
        ss = fmaf(h.v[i], h.v[i], ss);
}

// 1 / sqrt(mean of the squares + eps); 0 for a row of zeros, whose values are zero with any eps.
//
// Values and their scales are held `lift` times as large, a power of two, and
// the scales stored without it.  It is 1 up to eps = 2^60: h and the gains are at
// least 2^-24 where they are not 0 and h is at most 2^17, so the values are at
// least 2^-48 / (2^34 + eps)^(1/2) and the scales above 2^-90, as f8_quotient
// takes them.  With a larger eps 2^64 keeps them there.
__device__ __forceinline__ float norm_inverse(float ss, const NormArgs &a)
{
    return ss == 0.0f ? 0.0f : a.lift / sqrtf(ss / (float)a.K + a.eps);
}

__device__ __forceinline__ Eight norm_value(const Eight &h, uint4 gain, float inv)
{
    const Eight g = widen(gain);
    Eight y;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        y.v[i] = (h.v[i] * inv) * g.v[i];
    return y;
}

// The largest |v| as bits; a row whose squares' sum is not finite gives NaN.
__device__ __forceinline__ uint32_t norm_largest(const Eight &y, bool finite)
{
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        m = max(m, abs_bits(y.v[i]));
    return finite ? m : 0x7fc00000u;
}

template <NormOut OUT> __device__ __forceinline__ void norm_scale(uint32_t m, float &s, float &r)
{
    if (OUT == NormOut::F8) {
        f8_block_scale<false>(m, s, r);
        return;
    }
    s = m >= 0x7f800000u ? __uint_as_float(0x7fc00000u) : __uint_as_float(m) / 127.0f;
    s = s < 0x1p-126f ? 0.0f : s;
    r = s > 0.0f ? 1.0f / s : 0.0f;
}

template <NormOut OUT> __device__ __forceinline__ uint2 norm_codes(const Eight &y, float s, float r)
{
    if (OUT == NormOut::F8)
        return make_uint2(f8_codes4<false>(y.v[0], y.v[1], y.v[2], y.v[3], s, r),
                          f8_codes4<false>(y.v[4], y.v[5], y.v[6], y.v[7], s, r));
    return make_uint2(int8_codes4(y.v, s, r), int8_codes4(y.v + 4, s, r));
}

// Lanes that own a slice (eight values a lane), and where its scale goes.
template <NormOut OUT> constexpr int kSliceLanes = OUT == NormOut::INT8_64 ? 8 : 16;
template <NormOut OUT> __device__ __forceinline__ float *norm_scale_at(const NormArgs &a, int64_t row, int chunk)
{
    const int g = chunk / kSliceLanes<OUT>;
    return a.scale + (OUT == NormOut::F8 ? (int64_t)g * a.M + row : row * (int64_t)(a.K / (8 * kSliceLanes<OUT>)) + g);
}

__device__ __forceinline__ void norm_store_sum(const NormArgs &a, int64_t row, int c, const Eight &h)
{
    if (a.sum)
        reinterpret_cast<uint4 *>(a.sum + row * (int64_t)a.K)[c] =
            make_uint4(pack_h2(h.v[0], h.v[1]), pack_h2(h.v[2], h.v[3]), pack_h2(h.v[4], h.v[5]),
                       pack_h2(h.v[6], h.v[7]));
}

// A workgroup a row, as many waves as it fills with CPL chunks of eight values
// a lane, all in registers: the row is read once.  Its sum of squares and, for
// int8 rows, its largest value meet over the lanes and then in LDS.
//
// Bound by memory: 7 bytes a value with a residual, of which 4516 x 4096 take 27.5
// us into e4m3 (4.7 TB/s; a copy of 2 GiB runs at 4.95), 26.6 into int8 by rows and
// 27.5 by groups.  Without one, 3 bytes a value, 18.5 us (3.0 TB/s) and 19.2: a
// row's load, its meetings and its codes follow one another, and the vector
// unit is about half busy; a workgroup that has its next row's load on the way
// has not been tried.  Four waves a row in registers against one
// wave a row that reads it again for each step: 40.4 and 19.8 us, and 1 x 4096
// 9.3 against 3.5.
constexpr int kNormWaves = 16;
template <NormOut OUT, int CPL>
__global__ __launch_bounds__(64 * kNormWaves) void rmsnorm_quant_kernel(NormArgs a, int64_t first_row)
{
    __shared__ float sums[kNormWaves];
    __shared__ uint32_t tops[kNormWaves];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = (int)blockDim.x >> 6;
    const int64_t row = first_row + blockIdx.x;
    const int K = a.K, nch = K >> 3;
    const int first = (int)threadIdx.x;                    // chunk j of the lane: first + 64 waves j
    const uint4 *xr = reinterpret_cast<const uint4 *>(a.x + row * (int64_t)K);
    const uint4 *gr = reinterpret_cast<const uint4 *>(a.gain);
    const uint4 none = make_uint4(0u, 0u, 0u, 0u);
    Eight h[CPL];
    float ss = 0.0f;
    {
        uint4 x[CPL], r[CPL];
#pragma unroll
        for (int j = 0; j < CPL; ++j) {
            const int c = first + 64 * waves * j;
            x[j] = c < nch ? load_nt(xr + c) : none;
            r[j] = none;
        }
        if (a.residual) {
            const uint4 *rr = reinterpret_cast<const uint4 *>(a.residual + row * (int64_t)K);
#pragma unroll
            for (int j = 0; j < CPL; ++j) {
                const int c = first + 64 * waves * j;
                r[j] = c < nch ? load_nt(rr + c) : none;
            }
        }
#pragma unroll
        for (int j = 0; j < CPL; ++j) {
            h[j] = norm_sum(x[j], r[j]);
            norm_squares(h[j], ss);
        }
    }
    ss = wave_sum(ss);
    if (lane == 0)
        sums[wave] = ss;
    __syncthreads();
    ss = sums[0];
    for (int i = 1; i < waves; ++i)
        ss += sums[i];
    const float inv = norm_inverse(ss, a);
    const bool finite = ss < INFINITY;
    float s = 0.0f, r = 0.0f;
    if (OUT == NormOut::INT8_ROW) {
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < CPL; ++j) {
            const int c = first + 64 * waves * j;
            if (c < nch)
                norm_store_sum(a, row, c, h[j]);
            h[j] = norm_value(h[j], c < nch ? gr[c] : none, inv);
            top = max(top, norm_largest(h[j], finite));
        }
        top = group_max_u32<64>(top);
        if (lane == 0)
            tops[wave] = top;
        __syncthreads();
        for (int i = 0; i < waves; ++i)
            top = max(top, tops[i]);
        norm_scale<OUT>(top, s, r);
        if (threadIdx.x == 0)
            a.scale[row] = s * a.unlift;
    }
#pragma unroll
    for (int j = 0; j < CPL; ++j) {
        const int c = first + 64 * waves * j;
        if (OUT != NormOut::INT8_ROW) {
            if (c < nch)
                norm_store_sum(a, row, c, h[j]);
            h[j] = norm_value(h[j], c < nch ? gr[c] : none, inv);
            norm_scale<OUT>(group_max_u32<kSliceLanes<OUT>>(norm_largest(h[j], finite)), s, r);
            if (c < nch && lane % kSliceLanes<OUT> == 0)
                *norm_scale_at<OUT>(a, row, c) = s * a.unlift;
        }
        if (c < nch)
            reinterpret_cast<uint2 *>(a.q + row * (int64_t)K)[c] = norm_codes<OUT>(h[j], s, r);
    }
}

// Longer rows: one wavefront a row, which is read again for each step (from
// cache).  1 x 18432 26 us (1 x 16384, in registers, 5.2), 4516 x 20480 with a
// residual 237 (2.7 TB/s).  A lane sums up to 2^16 squares: eight at a time in
// fp32 and those in 64 bits, or the sum of 2^22 is off by up to 2e-3 of it.
template <NormOut OUT>
__global__ __launch_bounds__(256) void rmsnorm_quant_long_kernel(NormArgs a)
{
    const int lane = threadIdx.x & 63;
    const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (row >= a.M)
        return;
    const int K = a.K, nch = K >> 3;
    const uint4 *xr = reinterpret_cast<const uint4 *>(a.x + row * (int64_t)K);
    const uint4 *rr = a.residual ? reinterpret_cast<const uint4 *>(a.residual + row * (int64_t)K) : nullptr;
    const uint4 *gr = reinterpret_cast<const uint4 *>(a.gain);
    const uint4 none = make_uint4(0u, 0u, 0u, 0u);
    auto load = [&](int c) __attribute__((always_inline)) { return norm_sum(xr[c], rr ? rr[c] : none); };
    double total = 0.0;
    for (int c = lane; c < nch; c += 64) {
        float eight = 0.0f;
        norm_squares(load(c), eight);
        total += eight;
    }
    const float ss = (float)wave_sum(total);
    const float inv = norm_inverse(ss, a);
    const bool finite = ss < INFINITY;
    float s = 0.0f, r = 0.0f;
    if (OUT == NormOut::INT8_ROW) {
        uint32_t top = 0;
        for (int c = lane; c < nch; c += 64)
            top = max(top, norm_largest(norm_value(load(c), gr[c], inv), finite));
        norm_scale<OUT>(group_max_u32<64>(top), s, r);
        if (lane == 0)
            a.scale[row] = s * a.unlift;
    }
    for (int base = 0; base < nch; base += 64) {
        const int c = base + lane;
        Eight h{}, y{};
        if (c < nch) {
            h = load(c);
            y = norm_value(h, gr[c], inv);
        }
        if (OUT != NormOut::INT8_ROW) {
            norm_scale<OUT>(group_max_u32<kSliceLanes<OUT>>(norm_largest(y, finite)), s, r);
            if (c < nch && lane % kSliceLanes<OUT> == 0)
                *norm_scale_at<OUT>(a, row, c) = s * a.unlift;
        }
        if (c < nch) {
            reinterpret_cast<uint2 *>(a.q + row * (int64_t)K)[c] = norm_codes<OUT>(y, s, r);
            norm_store_sum(a, row, c, h);
        }
    }
}

template <NormOut OUT, int CPL> void launch_rows(const NormArgs &a, hipStream_t st)
{
    const unsigned waves = (a.K + 512 * CPL - 1) / (512 * CPL);
    // a launch of 2^32 threads would wrap
    constexpr int64_t kRowsALaunch = 1 << 21;
    for (int64_t row = 0; row < a.M; row += kRowsALaunch) {
        const int64_t rows = a.M - row < kRowsALaunch ? a.M - row : kRowsALaunch;
        hipLaunchKernelGGL((rmsnorm_quant_kernel<OUT, CPL>), dim3((unsigned)rows), dim3(64 * waves), 0, st, a, row);
    }
}

// One chunk a lane where rows are few (256 x 4096 5.3 us, with two 6.2) or
// short (4516 x 512 6.4 and 7.1), two where there are many (4516 x 4096 30.1 and
// 28.0, 4516 x 1024 10.8 and 10.1) or they need more than 16 waves.
template <NormOut OUT> void launch_norm(const NormArgs &a, hipStream_t st)
{
    const int K = a.K;
    if (K > 1024 * kNormWaves)
        hipLaunchKernelGGL(rmsnorm_quant_long_kernel<OUT>, dim3((unsigned)((a.M + 3) / 4)), dim3(256), 0, st, a);
    else if (K <= 512 || (a.M <= 1024 && K <= 512 * kNormWaves))
        launch_rows<OUT, 1>(a, st);
    else
        launch_rows<OUT, 2>(a, st);
}

}  // namespace

void launch_quantize_act_f8(const uint16_t *x, int64_t rows, int K, uint8_t *q, float *scale,
                            hipStream_t st)
{
    constexpr int64_t kWaves = 1 << 25;                    // of 64 threads; a launch of 2^32 threads would wrap
    int64_t waves = ((int64_t)K + 511) / 512;
    if (waves * rows > kWaves)
        waves = kWaves / rows;
    hipLaunchKernelGGL(quant_act_f8_kernel, dim3((unsigned)((rows * waves + 3) / 4)), dim3(256), 0, st, x, q, scale,
                       rows, K, (int)waves);
}

void launch_quantize_weight_f8(const uint16_t *w, int64_t N, int K, uint8_t *q, float *scale,
                               hipStream_t st)
{
    const int kblocks = (K + kF8Block - 1) / kF8Block;
    const int64_t nblocks = (N + kF8Block - 1) / kF8Block;
    hipLaunchKernelGGL(quant_weight_f8_kernel, dim3((unsigned)(nblocks * kblocks)), dim3(256), 0, st, w, q,
                       scale, N, K, kblocks);
}

void launch_rmsnorm_quant(NormOut out, NormArgs a, hipStream_t st)
{
    a.lift = a.eps > 0x1p60f ? kF8Lift : 1.0f;
    a.unlift = 1.0f / a.lift;
    switch (out) {
    case NormOut::INT8_ROW: launch_norm<NormOut::INT8_ROW>(a, st); return;
    case NormOut::INT8_64: launch_norm<NormOut::INT8_64>(a, st); return;
    case NormOut::INT8_128: launch_norm<NormOut::INT8_128>(a, st); return;
    case NormOut::F8: launch_norm<NormOut::F8>(a, st); return;
    }
}

}  // namespace w4a8

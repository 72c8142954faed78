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
    return make_uint2(f8_codes4(lo_h2f(v.x), hi_h2f(v.x), lo_h2f(v.y), hi_h2f(v.y), s, r),
                      f8_codes4(lo_h2f(v.z), hi_h2f(v.z), lo_h2f(v.w), hi_h2f(v.w), s, r));
}

// The largest |x| of fp16 values, as fp16 bits, to fp32 bits: infinities and
// NaN stay above every finite value.
__device__ __forceinline__ uint32_t amax_h2f_bits(uint32_t m) { return __float_as_uint(h2f((uint16_t)m)); }

// One wavefront a row; 16 lanes own a block of 128, 8 values a lane.
__global__ __launch_bounds__(256) void quant_act_f8_kernel(const uint16_t *__restrict__ x,
                                                           uint8_t *__restrict__ q,
                                                           float *__restrict__ scale, int64_t rows,
                                                           int K)
{
    const int lane = threadIdx.x & 63;
    const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (row >= rows)
        return;
    const int nch = K >> 3;
    const uint4 *xr = reinterpret_cast<const uint4 *>(x + row * (int64_t)K);
    for (int base = 0; base < nch; base += 64) {
        const int c = base + lane;
        const bool valid = c < nch;
        const uint4 v = valid ? xr[c] : make_uint4(0u, 0u, 0u, 0u);
        const uint32_t m = group_max_u32<16>(absmax_bits8(v));
        float s, r;
        f8_block_scale(amax_h2f_bits(m), s, r);
        if (!valid)
            continue;
        if ((lane & 15) == 0)
            scale[(int64_t)(c >> 4) * rows + row] = s;
        reinterpret_cast<uint2 *>(q + row * (int64_t)K)[c] = f8_chunk8(v, s, r);
    }
}

// One workgroup a 128 x 128 block: wave w owns rows w, w + 4, ..., four rows a
// step (16 lanes each).
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
    f8_block_scale(amax_h2f_bits(m), s, r);
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

__device__ __forceinline__ float wave_sum(float v)
{
#pragma unroll
    for (int d = 32; d > 0; d >>= 1)
        v += __shfl_xor(v, d);
    return v;
}

// fl32(v / s) to an int8 code; v is no more than the slice's largest, but the
// quotient is taken in fp32, so it is clamped as the rule says.
__device__ __forceinline__ uint32_t int8_codes4(const float *v, float s, float r)
{
    int c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        c[i] = r == 0.0f ? 0 : quant_code_corrected(v[i], s, r, 127.0f);
    return pack_i8x4(c[0], c[1], c[2], c[3]);
}

// One wavefront a row, the row read three times (from cache after the first).
template <NormOut OUT>
__global__ __launch_bounds__(256) void rmsnorm_quant_kernel(NormArgs a)
{
    const int lane = threadIdx.x & 63;
    const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (row >= a.M)
        return;
    const int K = a.K, nch = K >> 3;
    const uint4 *xr = reinterpret_cast<const uint4 *>(a.x + row * (int64_t)K);
    const uint4 *rr = reinterpret_cast<const uint4 *>(a.residual + (a.residual ? row * (int64_t)K : 0));
    const uint4 *gr = reinterpret_cast<const uint4 *>(a.gain);
    auto load = [&](int c) __attribute__((always_inline)) {
        Eight h = widen(xr[c]);
        if (a.residual) {
            const Eight t = widen(rr[c]);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                h.v[i] += t.v[i];
        }
        return h;
    };
    float ss = 0.0f;
    for (int c = lane; c < nch; c += 64) {
        const Eight h = load(c);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            ss = fmaf(h.v[i], h.v[i], ss);
    }
    ss = wave_sum(ss);
    const float inv = 1.0f / sqrtf(ss / (float)K + a.eps);
    const bool finite = ss < INFINITY;
    auto normed = [&](const Eight &h, int c) __attribute__((always_inline)) {
        const Eight g = widen(gr[c]);
        Eight y;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            y.v[i] = ss == 0.0f ? 0.0f : (h.v[i] * inv) * g.v[i];
        return y;
    };
    auto largest = [&](const Eight &y) __attribute__((always_inline)) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            m = max(m, abs_bits(y.v[i]));
        return finite ? m : 0x7fc00000u;
    };
    constexpr float kMax = OUT == NormOut::F8 ? kF8Max : 127.0f;
    auto scale_of = [&](uint32_t m, float &s, float &r) __attribute__((always_inline)) {
        if (OUT == NormOut::F8) {
            f8_block_scale(m, s, r);
        } else {
            s = m >= 0x7f800000u ? __uint_as_float(0x7fc00000u) : __uint_as_float(m) / kMax;
            s = s < 0x1p-126f ? 0.0f : s;
            r = s > 0.0f ? 1.0f / s : 0.0f;
        }
    };
    uint32_t row_max = 0;
    float s = 0.0f, r = 0.0f;
    if (OUT == NormOut::INT8_ROW) {
        for (int c = lane; c < nch; c += 64)
            row_max = max(row_max, largest(normed(load(c), c)));
        scale_of(group_max_u32<64>(row_max), s, r);
        if (lane == 0)
            a.scale[row] = s;
    }
    for (int base = 0; base < nch; base += 64) {
        const int c = base + lane;
        const bool valid = c < nch;
        Eight h{}, y{};
        if (valid) {
            h = load(c);
            y = normed(h, c);
        }
        if (OUT != NormOut::INT8_ROW) {
            constexpr int kLanes = OUT == NormOut::INT8_64 ? 8 : 16;
            scale_of(group_max_u32<kLanes>(valid ? largest(y) : 0u), s, r);
            if (valid && lane % kLanes == 0) {
                const int g = c / kLanes;
                if (OUT == NormOut::F8)
                    a.scale[(int64_t)g * a.M + row] = s;
                else
                    a.scale[row * (int64_t)(nch / kLanes) + g] = s;
            }
        }
        if (!valid)
            continue;
        uint2 codes;
        if (OUT == NormOut::F8)
            codes = make_uint2(f8_codes4(y.v[0], y.v[1], y.v[2], y.v[3], s, r),
                               f8_codes4(y.v[4], y.v[5], y.v[6], y.v[7], s, r));
        else
            codes = make_uint2(int8_codes4(y.v, s, r), int8_codes4(y.v + 4, s, r));
        reinterpret_cast<uint2 *>(a.q + row * (int64_t)K)[c] = codes;
        if (a.sum)
            reinterpret_cast<uint4 *>(a.sum + row * (int64_t)K)[c] =
                make_uint4(pack_h2(h.v[0], h.v[1]), pack_h2(h.v[2], h.v[3]), pack_h2(h.v[4], h.v[5]),
                           pack_h2(h.v[6], h.v[7]));
    }
}

}  // namespace


void launch_quantize_act_f8(const uint16_t *x, int64_t rows, int K, uint8_t *q, float *scale,
                            hipStream_t st)
{
    hipLaunchKernelGGL(quant_act_f8_kernel, dim3((unsigned)((rows + 3) / 4)), dim3(256), 0, st, x, q, scale,
                       rows, K);
}

void launch_quantize_weight_f8(const uint16_t *w, int64_t N, int K, uint8_t *q, float *scale,
                               hipStream_t st)
{
    const int kblocks = (K + kF8Block - 1) / kF8Block;
    const int64_t nblocks = (N + kF8Block - 1) / kF8Block;
    hipLaunchKernelGGL(quant_weight_f8_kernel, dim3((unsigned)(nblocks * kblocks)), dim3(256), 0, st, w, q,
                       scale, N, K, kblocks);
}

void launch_rmsnorm_quant(NormOut out, const NormArgs &a, hipStream_t st)
{
    const dim3 grid((unsigned)((a.M + 3) / 4)), block(256);
    switch (out) {
    case NormOut::INT8_ROW: hipLaunchKernelGGL(rmsnorm_quant_kernel<NormOut::INT8_ROW>, grid, block, 0, st, a); return;
    case NormOut::INT8_64: hipLaunchKernelGGL(rmsnorm_quant_kernel<NormOut::INT8_64>, grid, block, 0, st, a); return;
    case NormOut::INT8_128: hipLaunchKernelGGL(rmsnorm_quant_kernel<NormOut::INT8_128>, grid, block, 0, st, a); return;
    case NormOut::F8: hipLaunchKernelGGL(rmsnorm_quant_kernel<NormOut::F8>, grid, block, 0, st, a); return;
    }
}

}  // namespace w4a8

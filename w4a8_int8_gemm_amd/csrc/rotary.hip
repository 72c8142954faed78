// Rotary positions with one to three axes on rows of heads (include/w4a8.h:
// rotary_axes).
//
// Per token the pairs' angles are formed once for all heads: in fp64, since
// a far position times a frequency loses the fraction of a turn in fp32
// (10^6 * 2^-24 = 0.06 rad); reduced to a turn there, cosine and sine in fp32
// (sincospif of the fraction).  Bound by memory: 2 bytes read and 2 written per
// element.  4516 tokens of 40 heads of 128, 92.6 MB: 15.6 us; one token: 2.5 us,
// about an empty launch.
#include "kv4.hpp"

namespace w4a8 {

namespace {

struct Sections {
    int axes;
    int n[3];
    int interleaved;
};

// Axis of pair i.
__device__ __forceinline__ int axis_of(const Sections &s, int i)
{
    if (s.interleaved) {
        const int a = i % s.axes;
        return i / s.axes < s.n[a] ? a : 0;
    }
    return i < s.n[0] ? 0 : i < s.n[0] + s.n[1] ? 1 : 2;
}

constexpr int kMaxHalf = 512;
constexpr int64_t kGridRow = 1 << 22;       // tokens along x: a dimension of a grid has under 2^32 threads

__global__ __launch_bounds__(256) void rotary_kernel(const uint16_t *x, int64_t x_stride,
                                                     const int64_t *__restrict__ pos,
                                                     const float *__restrict__ inv_freq, int64_t T,
                                                     int heads, int D, int R, Sections sec,
                                                     uint16_t *out, int64_t out_stride)
{
    __shared__ float cs[kMaxHalf], sn[kMaxHalf];
    const int64_t t = blockIdx.y * kGridRow + blockIdx.x;
    if (t >= T)
        return;
    const int half = R / 2;
    for (int i = threadIdx.x; i < half; i += 256) {
        const double turns = (double)pos[axis_of(sec, i) * T + t] * (double)inv_freq[i] *
                             0.15915494309189533577;      // 1 / (2 pi)
        const float f = (float)(turns - rint(turns));
        float c, s;
        sincospif(2.0f * f, &s, &c);
        cs[i] = c;
        sn[i] = s;
    }
    __syncthreads();
    const int pairs = half / 8, rest = (D - R) / 8, per = pairs + rest;   // 16-byte pieces
    for (int w = threadIdx.x; w < heads * per; w += 256) {
        const int h = w / per, c = w % per;
        const uint16_t *src = x + t * x_stride + (int64_t)h * D;
        uint16_t *dst = out + t * out_stride + (int64_t)h * D;
        if (c >= pairs) {
            const int at = R + (c - pairs) * 8;
            *reinterpret_cast<uint4 *>(dst + at) = *reinterpret_cast<const uint4 *>(src + at);
            continue;
        }
        const uint4 a4 = *reinterpret_cast<const uint4 *>(src + c * 8);
        const uint4 b4 = *reinterpret_cast<const uint4 *>(src + half + c * 8);
        const uint32_t a[4] = {a4.x, a4.y, a4.z, a4.w}, b[4] = {b4.x, b4.y, b4.z, b4.w};
        uint32_t u[4], v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float c0 = cs[c * 8 + 2 * j], s0 = sn[c * 8 + 2 * j];
            const float c1 = cs[c * 8 + 2 * j + 1], s1 = sn[c * 8 + 2 * j + 1];
            const float a0 = lo_h2f(a[j]), a1 = hi_h2f(a[j]), b0 = lo_h2f(b[j]), b1 = hi_h2f(b[j]);
            u[j] = pack_h2(fmaf(a0, c0, -(b0 * s0)), fmaf(a1, c1, -(b1 * s1)));
            v[j] = pack_h2(fmaf(b0, c0, a0 * s0), fmaf(b1, c1, a1 * s1));
        }
        *reinterpret_cast<uint4 *>(dst + c * 8) = make_uint4(u[0], u[1], u[2], u[3]);
        *reinterpret_cast<uint4 *>(dst + half + c * 8) = make_uint4(v[0], v[1], v[2], v[3]);
    }
}

}  // namespace

void launch_rotary(const uint16_t *x, int64_t x_stride, const int64_t *pos, const float *inv_freq,
                   int64_t T, int heads, int D, int R, int axes, const int *sections,
                   bool interleaved, uint16_t *out, int64_t out_stride, hipStream_t st)
{
    Sections s;
    s.axes = axes;
    for (int a = 0; a < 3; ++a)
        s.n[a] = a < axes ? sections[a] : 0;
    s.interleaved = interleaved ? 1 : 0;
    const dim3 grid((unsigned)(T < kGridRow ? T : kGridRow), (unsigned)((T + kGridRow - 1) / kGridRow));
    hipLaunchKernelGGL(rotary_kernel, grid, dim3(256), 0, st, x, x_stride, pos,
                       inv_freq, T, heads, D, R, s, out, out_stride);
}

}  // namespace w4a8

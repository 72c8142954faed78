// Attention of few query rows over the 4-bit cache (include/w4a8.h:
// kv4_attention): up to 64 rows (queries x query heads of a kv head; 32 where
// head_dim is 256, whose outputs fill the registers) a sequence and kv head,
// so that the cache is read once.
//
// What bounds it: HBM.  A key and value of one head take D + 8 D / G bytes
// and 4 D operations per query row.
//
// One wavefront takes steps of 32 keys.  S^T = K Q^T on 16x16x32 matrix
// instructions with the codes as fp16 (exact) and the keys' scales applied to
// the fp32 scores; the result leaves a lane with one query row and four
// consecutive keys of each 16, which is, for two pieces of 16, the operand of
// the second product O^T = V^T P^T as it stands.  The cache's byte order
// gives a lane its operand bytes side by side: K's as one load of D / 8
// bytes, V's as D / 32 bytes of each of its eight keys.  The next step's
// loads are in flight while one is computed.
//
// The work is split in units of steps, the same number for every workgroup
// whatever the sequences' lengths: a workgroup finds its range of (sequence,
// head, step) from a scan of the lengths, splits each piece of it over its
// four waves and joins them in LDS.  Where a (sequence, head) lies in several
// workgroups' ranges each leaves its part in the workspace and the last to
// arrive joins them in order, so the result does not depend on who that is.
#include "kv4_device.hpp"

namespace w4a8 {

namespace {

constexpr int kWaves = 4;

struct Partial {
    float *base;                // [2 parts][slot_rows][D + 2]
    int slot_rows;
    uint64_t *counters;         // [B * heads]
    int parts, least;
    int row_limit;              // sequences with more rows are left to the other kernel
};

// What a lane loads for a step of 32 keys: pieces p = 0, 1 of 16 keys.  Of the
// scales, which the 16 lanes of a row share, a lane takes one key's: lane
// 8 p + 4 v + j of a row K's (v = 0) or V's (v = 1) of key 4 (lane / 16) + j.
template <int N32, int NG> struct Step {
    uint32_t k[2][N32];                 // key lane % 16: dims 32 i + 8 (lane / 16) ..+7
    uint32_t v[2][4][(N32 + 3) / 4];    // keys 4 (lane / 16) + j: dims 32 g + 2 (lane % 16) ..+1
    float sc[NG];
    bool ok[2];                         // the page exists
};

template <int D, int NG>
__device__ __forceinline__ void load_step(Step<D / 32, NG> &s, const Kv4Cache &c, int head, int page0, int page1,
                                          int step, int lane)
{
    constexpr int N32 = D / 32;
    const int r = lane & 15, b = lane >> 4;
    int64_t rows[2];
#pragma unroll
    for (int p = 0; p < 2; ++p) {
        const int page = p ? page1 : page0;
        s.ok[p] = kv4_page_ok(page, c.pages);
        const int at = (step * 32 + p * 16) & ((1 << c.shift) - 1);
        const int64_t row = rows[p] = c.row(s.ok[p] ? page : 0, head, at);
        const uint8_t *kp = c.k + row * (D / 2) + (uint32_t)(r * (D / 2) + b * (D / 8));
        const uint8_t *vp = c.v + row * (D / 2) + (uint32_t)(4 * b * (D / 2) + r * N32);
        if constexpr (N32 == 2) {
            const uint2 w = *reinterpret_cast<const uint2 *>(kp);
            s.k[p][0] = w.x, s.k[p][1] = w.y;
        } else {
#pragma unroll
            for (int i = 0; i < N32 / 4; ++i) {
                const v4u w = reinterpret_cast<const v4u *>(kp)[i];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    s.k[p][4 * i + e] = w[e];
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint8_t *q = vp + j * (D / 2);
            if constexpr (N32 == 2) {
                s.v[p][j][0] = *reinterpret_cast<const uint16_t *>(q);
            } else if constexpr (N32 == 4) {
                s.v[p][j][0] = *reinterpret_cast<const uint32_t *>(q);
            } else {
                const uint2 w = *reinterpret_cast<const uint2 *>(q);
                s.v[p][j][0] = w.x, s.v[p][j][1] = w.y;
            }
        }
    }
    const float *base = (r & 4) ? c.vs : c.ks;
    const float *sp = base + ((r & 8) ? rows[1] : rows[0]) * NG + (4 * b + (r & 3)) * NG;
    if constexpr (NG == 1) {
        s.sc[0] = *sp;
    } else if constexpr (NG == 2) {
        const float2 w = *reinterpret_cast<const float2 *>(sp);
        s.sc[0] = w.x, s.sc[1] = w.y;
    } else {
        const v4f w = *reinterpret_cast<const v4f *>(sp);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            s.sc[e] = w[e];
    }
}

template <int D, int NG, int RT>
__global__ __launch_bounds__(64 * kWaves, RT == 4 || RT * D == 512 ? 1 : 2) void kv4_decode_kernel(Kv4Cache c, Kv4AttnArgs a, Partial w)
{
    constexpr int N32 = D / 32, PER = N32 / NG;          // steps of 32 dims, of one group
    constexpr int LD = D + 4;                            // LDS row: 16 rows of float4 without bank conflicts
    __shared__ float os[kWaves][16][LD];
    __shared__ float refs[kWaves][16 * RT], ls[kWaves][16 * RT];
    __shared__ int last;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, b4 = lane >> 4;
    const int group = a.group, B = a.B;

    // ---- this workgroup's units
    const auto steps_of = [&](int b, Kv4Seq &s) {
        s = kv4_sequence(a, c.shift, b);
        return (int64_t)s.m * group > w.row_limit ? 0 : kv4_steps(s, a.causal, a.window).count;
    };
    int64_t total = 0;
    for (int base = 0; base < B; base += 64) {
        Kv4Seq s;
        int64_t n = base + lane < B ? steps_of(base + lane, s) : 0;
        for (int i = 32; i; i >>= 1)
            n += __shfl_xor(n, i);
        total += n;
    }
    total = uniform(total);
    const int64_t U = total * c.heads;
    if (U == 0)
        return;
    const int parts = kv4_parts(U, w.parts, w.least);
    if ((int)blockIdx.x >= parts)
        return;
    int64_t u = kv4_part_begin(U, parts, blockIdx.x);
    const int64_t u_end = kv4_part_begin(U, parts, blockIdx.x + 1);
    // the sequence that holds unit u, and the units before it
    int b = 0;
    int64_t before = 0;                                  // steps of the sequences before b
    for (int base = 0; base < B; base += 64) {
        Kv4Seq s;
        const int64_t n = base + lane < B ? steps_of(base + lane, s) : 0;
        int64_t inc = n;
        for (int i = 1; i < 64; i <<= 1) {
            const int64_t up = __shfl_up(inc, i);
            inc += lane >= i ? up : 0;
        }
        const int64_t here = __shfl(inc, 63);
        if ((before + here) * c.heads > u) {
            const int at = __ffsll((unsigned long long)__ballot((before + inc) * c.heads > u)) - 1;
            before += __shfl(inc - n, at);
            b = base + at;
            break;
        }
        before += here;
    }
    before = uniform(before);
    b = __builtin_amdgcn_readfirstlane(b);

    while (u < u_end) {
        Kv4Seq seq;
        const int count = (int)steps_of(b, seq);
        if (count == 0) {
            ++b;
            continue;
        }
        const int64_t item0 = before * c.heads;          // the sequence's first unit
        const int head = (int)((u - item0) / count), s0 = (int)((u - item0) % count);
        const int64_t left = u_end - u;
        const int s1 = left < count - s0 ? s0 + (int)left : count;
        const Kv4Steps all = kv4_steps(seq, a.causal, a.window);
        const int rows = seq.m * group;

        // ---- queries: row lane % 16 of each 16, visible keys [lo, hi)
        h8 q[RT][N32];
        int lo[RT], hi[RT];
        float ref[RT], top[RT], l[RT];
        v4f o[RT][2 * N32];
        int lo_most = 0, hi_least = 0x7fffffff;
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            const int row = 16 * t + r;
            const int rc = row < rows ? row : rows - 1;  // rows past the last repeat it and are not stored
            const int i = rc / group, hh = rc % group;
            const uint16_t *qp = a.q + (int64_t)(seq.q0 + i) * a.q_stride + (int64_t)(head * group + hh) * D + 8 * b4;
#pragma unroll
            for (int k = 0; k < N32; ++k)
                q[t][k] = order8(*reinterpret_cast<const uint4 *>(qp + 32 * k));
            lo[t] = kv4_lo(seq.n, seq.m, i, a.window);
            hi[t] = kv4_hi(seq.n, seq.m, i, a.causal);
            ref[t] = 0.0f;
            top[t] = -INFINITY;
            l[t] = 0.0f;
#pragma unroll
            for (int k = 0; k < 2 * N32; ++k)
                o[t][k] = (v4f){0.0f, 0.0f, 0.0f, 0.0f};
        }
        lo_most = kv4_lo(seq.n, seq.m, seq.m - 1, a.window);
        hi_least = kv4_hi(seq.n, seq.m, 0, a.causal);
        int scale_exp = kNoScale;

        // ---- this wave's steps
        const int n = s1 - s0;
        const int w0 = all.first + s0 + n * wave / kWaves, w1 = all.first + s0 + n * (wave + 1) / kWaves;
        const int32_t *table = a.table + (int64_t)b * a.max_pages;
        const int last_page = seq.n > 0 ? (seq.n - 1) >> c.shift : -1;
        // pages of 64 pieces of 16 keys from `piece0`, one a lane; -1 past the last key
        int piece0 = 2 * w0;
        const auto pages_from = [&](int piece) {
            const int p = (int)(((int64_t)(piece + lane) * 16) >> c.shift);
            return p <= last_page ? table[p] : -1;
        };
        int pages = w0 < w1 ? pages_from(piece0) : -1;
        const auto fetch = [&](Step<N32, NG> &s, int step) {
            if (2 * step - piece0 >= 64) {
                piece0 = 2 * step;
                pages = pages_from(piece0);
            }
            load_step<D, NG>(s, c, head, __builtin_amdgcn_readlane(pages, 2 * step - piece0),
                             __builtin_amdgcn_readlane(pages, 2 * step - piece0 + 1), step, lane);
        };
        Step<N32, NG> next;
        if (w0 < w1)
            fetch(next, w0);
        for (int step = w0; step < w1; ++step) {
            Step<N32, NG> cur = next;
            if (step + 1 < w1)
                fetch(next, step + 1);
            const int t0 = step * 32;
            // scores
            float ksc[NG];
#pragma unroll
            for (int g = 0; g < NG; ++g)
                ksc[g] = cur.sc[g] * (a.scale * kLog2e);
            float s[RT][2][4];
            each<2>([&](auto pc) {
                constexpr int p = decltype(pc)::value;
                each<NG>([&](auto gc) {
                    constexpr int g = decltype(gc)::value;
                    v4f acc[RT];
#pragma unroll
                    for (int t = 0; t < RT; ++t)
                        acc[t] = (v4f){0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int k = g * PER; k < (g + 1) * PER; ++k) {
                        const h8 kk = codes8(cur.k[p][k]);
#pragma unroll
                        for (int t = 0; t < RT; ++t)
                            acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kk, q[t][k], acc[t], 0, 0, 0);
                    }
                    each<4>([&](auto jc) {
                        constexpr int j = decltype(jc)::value;
                        const float f = row_lane<8 * p + j>(ksc[g]);
#pragma unroll
                        for (int t = 0; t < RT; ++t)
                            s[t][p][j] = g == 0 ? acc[t][j] * f : fmaf(acc[t][j], f, s[t][p][j]);
                    });
                });
            });
            // a step that not every row sees whole: hide keys, and what garbage stands for them
            if (!cur.ok[0] || !cur.ok[1] || t0 < lo_most || t0 > hi_least - 32) {
#pragma unroll
                for (int p = 0; p < 2; ++p) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int key = t0 + 16 * p + 4 * b4 + j;
                        const bool there = cur.ok[p] && key < seq.n;
#pragma unroll
                        for (int t = 0; t < RT; ++t)
                            s[t][p][j] = there && key >= lo[t] && key < hi[t] ? s[t][p][j] : -INFINITY;
                    }
                }
                const int mine = t0 + 2 * (r & 8) + 4 * b4 + (r & 3);
                const bool there = ((r & 8) ? cur.ok[1] : cur.ok[0]) && mine < seq.n;
#pragma unroll
                for (int g = 0; g < NG; ++g)
                    cur.sc[g] = there ? cur.sc[g] : 0.0f;
            }
            // the largest value scale so far
            float big = cur.sc[0];
#pragma unroll
            for (int g = 1; g < NG; ++g)
                big = fmaxf(big, cur.sc[g]);
            big = (r & 4) ? big : 0.0f;
            big = max_rows(__uint_as_float(group_max_u32<16>(__float_as_uint(big))));
            scale_exp = max(scale_exp, __builtin_amdgcn_readfirstlane(exponent_of(big)));
            const float shift = (float)(scale_exp - kHeadroom);
            h8 wt[RT][NG];
#pragma unroll
            for (int t = 0; t < RT; ++t) {
                float m = fmaxf(fmaxf(fmaxf(s[t][0][0], s[t][0][1]), fmaxf(s[t][0][2], s[t][0][3])),
                                fmaxf(fmaxf(s[t][1][0], s[t][1][1]), fmaxf(s[t][1][2], s[t][1][3])));
                m = fmaxf(top[t], max_rows(m));
                const float nref = (m == -INFINITY ? 0.0f : m) + shift;
                if (__ballot(nref != ref[t])) {          // rare after the first steps
                    const float alpha = top[t] == -INFINITY ? 0.0f : exp2_hw(ref[t] - nref);
                    l[t] *= alpha;
#pragma unroll
                    for (int k = 0; k < 2 * N32; ++k)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            o[t][k][e] *= alpha;
                    ref[t] = nref;
                }
                top[t] = m;
#pragma unroll
                for (int p = 0; p < 2; ++p)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        s[t][p][j] = exp2_hw(s[t][p][j] - nref);
                        l[t] += s[t][p][j];
                    }
                // weight times the value's scale, the one rounding to fp16
                each<NG>([&](auto gc) {
                    constexpr int g = decltype(gc)::value;
                    u32x4 x;
                    each<4>([&](auto ic) {
                        constexpr int p = decltype(ic)::value / 2, j = decltype(ic)::value % 2 * 2;
                        x[2 * p + j / 2] = pack_h2(s[t][p][j] * row_lane<8 * p + 4 + j>(cur.sc[g]),
                                                   s[t][p][j + 1] * row_lane<8 * p + 5 + j>(cur.sc[g]));
                    });
                    wt[t][g] = __builtin_bit_cast(h8, x);
                });
            }
            // O^T += V^T P^T: 16 rows 32 g + 2 r + e of the values for byte g's two nibbles e
            each<N32>([&](auto gc) {
                constexpr int g = decltype(gc)::value;
                const uint32_t x0 = byte_pair<g % 4>(cur.v[0][0][g / 4], cur.v[0][1][g / 4]);
                const uint32_t x1 = byte_pair<g % 4>(cur.v[0][2][g / 4], cur.v[0][3][g / 4]);
                const uint32_t x2 = byte_pair<g % 4>(cur.v[1][0][g / 4], cur.v[1][1][g / 4]);
                const uint32_t x3 = byte_pair<g % 4>(cur.v[1][2][g / 4], cur.v[1][3][g / 4]);
                const u32x4 e0 = {codes_low(x0), codes_low(x1), codes_low(x2), codes_low(x3)};
                const u32x4 e1 = {codes_high(x0), codes_high(x1), codes_high(x2), codes_high(x3)};
#pragma unroll
                for (int t = 0; t < RT; ++t) {
                    o[t][2 * g] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, e0), wt[t][g / PER],
                                                                         o[t][2 * g], 0, 0, 0);
                    o[t][2 * g + 1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, e1), wt[t][g / PER],
                                                                             o[t][2 * g + 1], 0, 0, 0);
                }
            });
        }

        // ---- join the four waves
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            l[t] = sum_rows(l[t]);
            if (lane < 16) {
                refs[wave][16 * t + r] = l[t] > 0.0f ? ref[t] : -INFINITY;
                ls[wave][16 * t + r] = l[t];
            }
        }
        __syncthreads();
        const bool whole = s0 == 0 && s1 == count;
        const int64_t item = (int64_t)b * c.heads + head;
        const int64_t first_unit = item0 + (int64_t)head * count;
        // a part that does not begin its item is its workgroup's first
        float *slot = w.base + (int64_t)(2 * blockIdx.x + (s0 == 0 ? 1 : 0)) * w.slot_rows * (D + 2);
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            if (16 * t >= rows)
                break;
            float R = -INFINITY;
#pragma unroll
            for (int x = 0; x < kWaves; ++x)
                R = fmaxf(R, refs[x][16 * t + r]);
            const float f = l[t] > 0.0f ? exp2_hw(ref[t] - R) : 0.0f;
#pragma unroll
            for (int g = 0; g < N32; ++g) {
                // lane: dims 32 g + 8 b4 + 2 reg + e
                float4 x, y;
                x.x = o[t][2 * g][0] * f, x.y = o[t][2 * g + 1][0] * f, x.z = o[t][2 * g][1] * f, x.w = o[t][2 * g + 1][1] * f;
                y.x = o[t][2 * g][2] * f, y.y = o[t][2 * g + 1][2] * f, y.z = o[t][2 * g][3] * f, y.w = o[t][2 * g + 1][3] * f;
                float4 *dst = reinterpret_cast<float4 *>(&os[wave][r][32 * g + 8 * b4]);
                dst[0] = x;
                dst[1] = y;
            }
            __syncthreads();
            // a thread: four dims of a row at a time
            for (int x = threadIdx.x; x < 16 * (D / 4); x += 64 * kWaves) {
                const int rr = x / (D / 4), d = x % (D / 4) * 4, row = 16 * t + rr;
                if (row >= rows)
                    continue;
                float RR = -INFINITY, L = 0.0f;
#pragma unroll
                for (int y = 0; y < kWaves; ++y)
                    RR = fmaxf(RR, refs[y][row]);
#pragma unroll
                for (int y = 0; y < kWaves; ++y)
                    L += ls[y][row] > 0.0f ? ls[y][row] * exp2_hw(refs[y][row] - RR) : 0.0f;
                float4 sum = *reinterpret_cast<const float4 *>(&os[0][rr][d]);
#pragma unroll
                for (int y = 1; y < kWaves; ++y) {
                    const float4 v = *reinterpret_cast<const float4 *>(&os[y][rr][d]);
                    sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
                }
                if (whole) {
                    const float inv = L > 0.0f ? 1.0f / L : 0.0f;
                    const int64_t at = (int64_t)(seq.q0 + row / group) * a.q_heads + head * group + row % group;
                    *reinterpret_cast<uint2 *>(a.out + at * D + d) =
                        make_uint2(pack_h2(sum.x * inv, sum.y * inv), pack_h2(sum.z * inv, sum.w * inv));
                    if (a.lse && d == 0)
                        a.lse[at] = L > 0.0f ? (RR + __builtin_amdgcn_logf(L)) * kLn2 : -INFINITY;
                } else {
                    float *dst = slot + (int64_t)row * (D + 2);
                    store_shared(dst + d, sum.x, sum.y);
                    store_shared(dst + d + 2, sum.z, sum.w);
                    if (d == 0)
                        store_shared(dst + D, RR, L);
                }
            }
            __syncthreads();
        }
        if (!whole) {
            // ---- join the workgroups: the last to arrive reads all parts in order
            const int64_t last_unit = first_unit + count - 1;
            const int p0 = kv4_part_of(U, parts, first_unit), p1 = kv4_part_of(U, parts, last_unit);
            __builtin_amdgcn_s_waitcnt(0);               // this wave's parts are stored
            __syncthreads();
            if (threadIdx.x == 0)
                last = arrive_last(w.counters + item, a.tag, p1 - p0 + 1) ? 1 : 0;
            __syncthreads();
            if (last) {
                for (int x = threadIdx.x; x < rows * (D / 4); x += 64 * kWaves) {
                    const int row = x / (D / 4), d = x % (D / 4) * 4;
                    const auto part = [&](int p) {
                        const int second = p == p0 ? 1 : 0;
                        return w.base + ((int64_t)(2 * p + second) * w.slot_rows + row) * (D + 2);
                    };
                    float RR = -INFINITY;
                    for (int p = p0; p <= p1; ++p) {
                        const float2 x2 = load_shared(part(p) + D);
                        RR = fmaxf(RR, x2.y > 0.0f ? x2.x : -INFINITY);
                    }
                    float L = 0.0f;
                    float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    for (int p = p0; p <= p1; ++p) {
                        const float2 rl = load_shared(part(p) + D), x0 = load_shared(part(p) + d), x1 = load_shared(part(p) + d + 2);
                        const float f = rl.y > 0.0f ? exp2_hw(rl.x - RR) : 0.0f;
                        L = fmaf(rl.y, f, L);
                        sum.x = fmaf(x0.x, f, sum.x), sum.y = fmaf(x0.y, f, sum.y);
                        sum.z = fmaf(x1.x, f, sum.z), sum.w = fmaf(x1.y, f, sum.w);
                    }
                    const float inv = L > 0.0f ? 1.0f / L : 0.0f;
                    const int64_t at = (int64_t)(seq.q0 + row / group) * a.q_heads + head * group + row % group;
                    *reinterpret_cast<uint2 *>(a.out + at * D + d) =
                        make_uint2(pack_h2(sum.x * inv, sum.y * inv), pack_h2(sum.z * inv, sum.w * inv));
                    if (a.lse && d == 0)
                        a.lse[at] = L > 0.0f ? (RR + __builtin_amdgcn_logf(L)) * kLn2 : -INFINITY;
                }
            }
            __syncthreads();                             // `last` is read before it is written again
        }
        u += s1 - s0;
        if (u == item0 + (int64_t)c.heads * count) {
            before += count;
            ++b;
        }
    }
}

template <int D, int NG>
void launch(const Kv4Cache &c, const Kv4AttnArgs &a, const Partial &w, int rows, hipStream_t st)
{
    const dim3 grid((unsigned)w.parts), block(64 * kWaves);
    if (rows <= 16)
        hipLaunchKernelGGL((kv4_decode_kernel<D, NG, 1>), grid, block, 0, st, c, a, w);
    else if (rows <= 32)
        hipLaunchKernelGGL((kv4_decode_kernel<D, NG, 2>), grid, block, 0, st, c, a, w);
    else if constexpr (D < 256)
        hipLaunchKernelGGL((kv4_decode_kernel<D, NG, 4>), grid, block, 0, st, c, a, w);
}

}  // namespace

void launch_kv4_decode(const Kv4Cache &c, const Kv4AttnArgs &a, int rows, hipStream_t st)
{
    Partial w;
    w.parts = kDecodeParts;
    w.least = 16;
    w.row_limit = rows;
    w.slot_rows = rows;
    w.counters = static_cast<uint64_t *>(a.workspace);
    w.base = reinterpret_cast<float *>(static_cast<char *>(a.workspace) + kv4_counter_bytes(a.B, c.heads));
    switch (c.D * 8 + c.D / c.G) {
    case 64 * 8 + 1: launch<64, 1>(c, a, w, rows, st); return;
    case 64 * 8 + 2: launch<64, 2>(c, a, w, rows, st); return;
    case 128 * 8 + 1: launch<128, 1>(c, a, w, rows, st); return;
    case 128 * 8 + 2: launch<128, 2>(c, a, w, rows, st); return;
    case 128 * 8 + 4: launch<128, 4>(c, a, w, rows, st); return;
    case 256 * 8 + 1: launch<256, 1>(c, a, w, rows, st); return;
    case 256 * 8 + 2: launch<256, 2>(c, a, w, rows, st); return;
    default: launch<256, 4>(c, a, w, rows, st); return;
    }
}

}  // namespace w4a8

// Attention of many query rows over the 4-bit cache (include/w4a8.h:
// kv4_attention): sequences with more rows a kv head than the kernel for few
// rows takes.
//
// What bounds it: a wave's own chain of LDS reads, products and softmax, with
// two waves a SIMD to cover it.  For D = 128, a wave's tile of 64 keys and 32
// rows takes 32 matrix instructions and 424 vector instructions (scaling,
// maximum, exponential, sum, rounding, and its share of turning codes into
// fp16).  Of all cycles the vector unit is busy 57 %, the matrix unit 32 %: the
// two work almost one after the other.  Measured: a causal prompt of 4516
// tokens, 167 GFLOP, 222 to 232 us in different sessions (720 to 752 TFLOP/s).
//
// A workgroup has 128 rows (queries x query heads of one kv head), 32 a wave,
// and walks over its keys in tiles of 64.  Two of its waves turn the tile's V
// and two its K into fp16 in LDS (exact codes; the scales stay apart in fp32),
// while the next tile's codes are on their way.  S^T = K Q^T on 32x32x16
// matrix instructions leaves a lane with one query row and runs of four keys,
// which is the operand of O^T = V^T P^T if V^T's keys lie in that order: they
// do, eight keys of two such runs in one 16-byte piece.
//
// Where the rows alone do not fill the chip a (sequence, head, rows) tile's
// keys are cut into parts of equal width, joined as in the kernel for few rows.
#include "kv4_device.hpp"
#include "lds_copy.hpp"

namespace w4a8 {

namespace {

typedef float v16f __attribute__((ext_vector_type(16)));

constexpr uint32_t kNotThere = 0xffffffffu;             // bits of a value that is no number, one of many
__device__ __forceinline__ bool not_there(float k_scale) { return __float_as_uint(k_scale) == kNotThere; }

constexpr int kRows = kTileRows, kKeys = 64, kThreads = 2 * kRows;

template <int D, int NG>
__global__ __launch_bounds__(kThreads, D == 64 ? 3 : D < 256 ? 2 : 1) void kv4_prefill_kernel(Kv4Cache c, Kv4AttnArgs a, Partial w)
{
    constexpr int N32 = D / 32, PER = N32 / NG, KC = D / 8, VC = kKeys / 8;
    // a piece more in a row than it holds: 16 rows' pieces are on different banks
    __shared__ u32x4 kt[2][kKeys][KC + 1];               // fp16 codes [key][dim], pieces of 8 dims
    __shared__ u32x4 vt[2][D][VC + 1];                   // fp16 codes [dim][key], pieces of 8 keys
    __shared__ float ksc[2][NG][kKeys], vsc[2][NG][kKeys];
    __shared__ int last;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int group = a.group, B = a.B;

    // ---- this workgroup's tile of rows and part of the keys, as in the kernel
    // for few rows; the parts of a sequence's tiles are cut at the same keys
    Kv4Seq sl;
    int tl = 0, nl = 0;                                  // tiles of rows, steps of keys
    const auto lookup = [&](int base) {
        tl = nl = 0;
        if (base + lane < B) {
            sl = kv4_sequence(a, c.shift, base + lane);
            const int64_t rows = (int64_t)sl.m * group;
            if (rows > w.row_limit) {
                tl = (int)((rows + kRows - 1) / kRows);
                nl = kv4_steps(sl, a.causal, a.window, kKeys).count;
            }
        }
    };
    int64_t steps = 0;
    for (int base = 0; base < B; base += 64) {
        lookup(base);
        steps += wave_sum64((int64_t)tl * nl);
    }
    const int limit = kv4_tile_limit(steps * c.heads, kKeys);
    int b = -1, tiles = 0, cuts = 0, id = blockIdx.x, split = 0;   // split: slots before b's
    Kv4Seq seq = {0, 0, 0, 0};
    for (int base = 0; base < B; base += 64) {
        if (B > 64)
            lookup(base);
        const int k = tl ? (nl + limit - 1) / limit : 0;
        const int inc = prefix_sum(tl * k * c.heads), sinc = prefix_sum(k > 1 ? tl * k * c.heads : 0);
        const uint64_t past = __ballot(inc > id);
        if (past) {
            const int at = __builtin_ctzll(past);
            b = base + at;
            tiles = __builtin_amdgcn_readlane(tl, at);
            cuts = __builtin_amdgcn_readlane(k, at);
            seq.q0 = __builtin_amdgcn_readlane(sl.q0, at);
            seq.m = __builtin_amdgcn_readlane(sl.m, at);
            seq.n = __builtin_amdgcn_readlane(sl.n, at);
            seq.rest = __builtin_amdgcn_readlane(sl.rest, at);
            id -= __builtin_amdgcn_readlane(inc, at) - tiles * cuts * c.heads;
            split += cuts > 1 ? __builtin_amdgcn_readlane(sinc, at) - tiles * cuts * c.heads : 0;
            break;
        }
        id -= __builtin_amdgcn_readlane(inc, 63);
        split += __builtin_amdgcn_readlane(sinc, 63);
    }
    if (b < 0)
        return;
    // Head first, so that neighbours (other chiplets) have other heads' keys;
    // the last rows, which see the most keys, first.
    const int head = id % c.heads, part = id / c.heads % cuts, tile = tiles - 1 - id / c.heads / cuts;
    const int rows = seq.m * group, row0 = tile * kRows, rows_here = min(kRows, rows - row0);
    // the steps that some row of the tile sees, and the parts that hold any of them
    const int i_first = query_of(row0, w.over_group, group), i_last = query_of(row0 + rows_here - 1, w.over_group, group);
    const Kv4TilePart span = kv4_tile_part(seq, a.causal, a.window, kKeys, i_first, i_last,
                                           kv4_steps(seq, a.causal, a.window, kKeys), cuts, part);
    const int part0 = span.part0, parts = span.parts, s0 = span.s0, s1 = span.s1;
    if (part < part0 || part >= part0 + parts)
        return;
    // slots and counters of the sequence's tiles: [tile][head][part]
    const int tile_head = tile * c.heads + head;
    if (cuts > 1 && split + (tile_head + 1) * cuts > w.slots)
        return;                                          // only where q_starts gives rows to several sequences
    const int slot0 = split + tile_head * cuts + part0;
    uint64_t *counter = w.counters + (int64_t)(split + tile_head * cuts) * kCounterStride;
    if (parts > 1 && threadIdx.x == 0)
        announce(counter, a.tag);

    // ---- queries: row lane % 32 of the wave's 32
    const int r32 = lane & 31, h = lane >> 5;
    const int row = row0 + 32 * wave + r32;
    const int rc = min(row, rows - 1);
    const int qi = query_of(rc, w.over_group, group), hh = rc - qi * group;
    h8 q[D / 16];
    {
        const uint16_t *qp = a.q + (int64_t)(seq.q0 + qi) * a.q_stride + (int64_t)(head * group + hh) * D + 8 * h;
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
            q[k] = order8(*reinterpret_cast<const uint4 *>(qp + 16 * k));
    }
    const int lo = kv4_lo(seq, qi, a.window), hi = kv4_hi(seq, qi, a.causal);
    // of the wave's rows: keys that all see, keys that any sees
    const int wrow0 = min(row0 + 32 * wave, rows - 1), wrow1 = min(row0 + 32 * wave + 31, rows - 1);
    const int wi0 = query_of(wrow0, w.over_group, group), wi1 = query_of(wrow1, w.over_group, group);
    const int lo_any = kv4_lo(seq, wi0, a.window), lo_all = kv4_lo(seq, wi1, a.window);
    const int hi_all = kv4_hi(seq, wi0, a.causal), hi_any = kv4_hi(seq, wi1, a.causal);

    // ---- the producer's side of a thread
    const int32_t *table = a.table + (int64_t)b * a.max_pages;
    const int last_key = seq.n - 1;
    const bool for_v = wave < 2;
    const int u = threadIdx.x & 127;
    // V: 8 keys of piece u / 16 = (half of 32 keys, 16 of it, run), word u % 16; K: keys u / 4 and 32 more, words u % 4
    const int vkey = (u >> 5) * 16 + ((u >> 4) & 1) * 4;  // its keys: vkey + 0..3, vkey + 8 + 0..3
    const int pkey = for_v ? vkey : u >> 2;
    uint32_t code[8 * (N32 > 4 ? 2 : 1)];
    float scale[2][NG];
    int page[2];                                         // of the next tile's keys
    bool there[2] = {false, false};                      // the loaded tile's
    const auto pages_of = [&](int step) {
        const int k0 = min(step * kKeys + pkey, last_key), k1 = min(step * kKeys + pkey + (for_v ? 8 : 32), last_key);
        page[0] = table[k0 >> c.shift];
        page[1] = table[k1 >> c.shift];
    };
    const auto load_scales = [&](float (&s)[NG], const float *p) {
#pragma unroll
        for (int g = 0; g < NG; ++g)
            s[g] = p[g];
    };
    const auto fetch = [&](int step) {
        const int mask = (1 << c.shift) - 1;
        if (for_v) {
            const int r = u & 15, key = step * kKeys + vkey;
            const bool ok = kv4_page_ok(page[0], c.pages);
            const int64_t at = c.row(ok ? page[0] : 0, head, key & mask);
            const uint8_t *p = c.v + at * (D / 2) + r * N32;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint8_t *pj = p + (j % 4 + j / 4 * 8) * (D / 2);
                if constexpr (N32 == 2) {
                    code[j] = *reinterpret_cast<const uint16_t *>(pj);
                } else if constexpr (N32 == 4) {
                    code[j] = *reinterpret_cast<const uint32_t *>(pj);
                } else {
                    const uint2 x = *reinterpret_cast<const uint2 *>(pj);
                    code[2 * j] = x.x, code[2 * j + 1] = x.y;
                }
            }
            // lanes 0 .. 7 of a piece: its eight keys' scales
            const int mine = r % 4 + (r >> 2 & 1) * 8;
            there[0] = ok && key + mine <= last_key;
            load_scales(scale[0], c.vs + (at + mine) * NG);
        } else {
            const int b4 = u & 3;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int key = step * kKeys + (u >> 2) + 32 * x;
                const bool ok = kv4_page_ok(page[x], c.pages);
                const int64_t at = c.row(ok ? page[x] : 0, head, key & mask);
                there[x] = ok && key <= last_key;
                const uint8_t *p = c.k + at * (D / 2) + b4 * (D / 8);
                if constexpr (N32 == 2) {
                    const uint2 y = *reinterpret_cast<const uint2 *>(p);
                    code[2 * x] = y.x, code[2 * x + 1] = y.y;
                } else {
#pragma unroll
                    for (int i = 0; i < N32 / 4; ++i) {
                        const v4u y = reinterpret_cast<const v4u *>(p)[i];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            code[N32 * x + 4 * i + e] = y[e];
                    }
                }
                load_scales(scale[x], c.ks + at * NG);
            }
        }
    };
    // codes to LDS; a key that is not there has kNotThere for its first K scale, which
    // a key's own cannot be, and the V scale 0
    const auto produce = [&](auto bc) {
        constexpr int buf = decltype(bc)::value;
        if (for_v) {
            const int r = u & 15, piece = u >> 4;
            each<N32>([&](auto gc) {
                constexpr int g = decltype(gc)::value, W = N32 > 4 ? 2 : 1, o = g / 4;
                const uint32_t x0 = byte_pair<g % 4>(code[0 * W + o], code[1 * W + o]), x1 = byte_pair<g % 4>(code[2 * W + o], code[3 * W + o]);
                const uint32_t x2 = byte_pair<g % 4>(code[4 * W + o], code[5 * W + o]), x3 = byte_pair<g % 4>(code[6 * W + o], code[7 * W + o]);
                const int d = 32 * g + 2 * r;
                vt[buf][d][piece] = (u32x4){codes_low(x0), codes_low(x1), codes_low(x2), codes_low(x3)};
                vt[buf][d + 1][piece] = (u32x4){codes_high(x0), codes_high(x1), codes_high(x2), codes_high(x3)};
            });
            if (r < 8) {
#pragma unroll
                for (int g = 0; g < NG; ++g)
                    vsc[buf][g][vkey + r % 4 + (r >> 2) * 8] = there[0] ? scale[0][g] : 0.0f;
            }
        } else {
            const int b4 = u & 3;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int key = (u >> 2) + 32 * x;
#pragma unroll
                for (int i = 0; i < N32; ++i)
                    kt[buf][key][4 * i + b4] = __builtin_bit_cast(u32x4, codes8(code[N32 * x + i]));
                if (b4 == 0) {
#pragma unroll
                    for (int g = 1; g < NG; ++g)
                        ksc[buf][g][key] = scale[x][g];
                    const float own = not_there(scale[x][0]) ? NAN : scale[x][0];
                    ksc[buf][0][key] = there[x] ? own : __uint_as_float(kNotThere);
                }
            }
        }
    };

    // ---- the tiles
    v16f o[N32];
#pragma unroll
    for (int g = 0; g < N32; ++g)
#pragma unroll
        for (int e = 0; e < 16; ++e)
            o[g][e] = 0.0f;
    float ref = kFarBelow, bound = kFarBelow, l = 0.0f;
    int scale_exp = kNoScale;                            // of the largest value scale that the lane's row has seen
    uint32_t scale_cap = 0;                              // bits of 2^(e + 1) for the least of the rows' scale_exp
    uint32_t spoilt = 0;                                 // bit g: it has seen one of group g that is not finite
    const float score_scale = a.scale * kLog2e;
    // key of lane % 16 in the runs of four that the lane's half has of 32 keys
    const int lane_key = (lane & 15) / 4 * 8 + 4 * h + (lane & 3);
    // Scores of 32 keys: lane's row, keys 8 (e / 4) + 4 h + e % 4 of them.
    const auto products = [&](v16f &acc, auto xc, auto gc, auto bc) {
        constexpr int x = decltype(xc)::value, g = decltype(gc)::value, buf = decltype(bc)::value;
#pragma unroll
        for (int e = 0; e < 16; ++e)
            acc[e] = 0.0f;
#pragma unroll
        for (int k = g * 2 * PER; k < (g + 1) * 2 * PER; ++k)
            acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(h8, kt[buf][32 * x + r32][2 * k + h]), q[k], acc,
                                                         0, 0, 0);
    };
    const auto scale_scores = [&](float (&s)[16], const v16f &acc, float ks, auto gc) {
        each<16>([&](auto ec) {
            constexpr int e = decltype(ec)::value;
            const float f = row_lane<e>(ks);
            s[e] = decltype(gc)::value == 0 ? acc[e] * f : fmaf(acc[e], f, s[e]);
        });
    };
    const auto scores = [&](float (&s)[16], const float (&ks)[NG], auto xc, auto bc) {
        each<NG>([&](auto gc) {
            v16f acc;
            products(acc, xc, gc, bc);
            scale_scores(s, acc, ks[decltype(gc)::value], gc);
        });
    };
    const auto hide = [&](float (&s)[16], float ks0, int t0) {
        each<16>([&](auto ec) {
            constexpr int e = decltype(ec)::value;
            const int key = t0 + e / 4 * 8 + 4 * h + e % 4;
            const float there = row_lane<e>(ks0);        // by all lanes: no lane may be off when it is read
            s[e] = ((key >= lo) & (key < hi) & !not_there(there)) ? s[e] : -INFINITY;
        });
    };
    // The largest of a lane's scores.
    const auto largest = [&](const float (&s)[16]) {
        float m = max3(s[0], s[1], s[2]);
#pragma unroll
        for (int e = 3; e < 15; e += 2)
            m = max3(m, s[e], s[e + 1]);
        return max3(m, s[15], s[15]);
    };
    // A new reference for the rows that need one; s: weights that are not in the output yet.
    const auto rescale = [&](float m, float *s, int pending) {
        m = max_halves(m);
        if (m > bound) {
            const float nref = reference_for(ref, m, scale_exp);
            const float alpha = exp2_hw(ref - nref);     // 0 before the first key
            l *= alpha;
            ref = nref;
            bound = bound_for(ref, scale_exp);
#pragma unroll
            for (int g = 0; g < N32; ++g)
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    o[g][e] *= alpha;
#pragma unroll
            for (int i = 0; i < pending; ++i)
                s[i] *= alpha;
        }
    };
    const auto weights = [&](float (&s)[16]) {
        float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            s[e] = exp2_hw(s[e] - ref);
            sum[e % 4] += s[e];
        }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
    };
    // O^T += V^T P^T of 32 keys; weight times the value's scale, the one rounding
    // to fp16: an error of 2.9e-4 where fp32 weights leave 2.1e-4.  (What is left
    // of the weights in a second product for rows of few keys, as in the kernel
    // for few rows, does not fit in the registers: a prompt of 4516 tokens took
    // 261 us instead of 227, four of 1200 with G = 32 334 instead of 138.)
    const auto output = [&](const float (&s)[16], const float (&vs)[NG], auto xc, auto bc) {
        constexpr int x = decltype(xc)::value, buf = decltype(bc)::value;
        each<2>([&](auto mc) {
            constexpr int m2 = decltype(mc)::value;
            each<NG>([&](auto gc) {
                constexpr int grp = decltype(gc)::value;
                u32x4 y;
                each<4>([&](auto ic) {
                    constexpr int e = 8 * m2 + 2 * decltype(ic)::value;
                    y[decltype(ic)::value] = pack_h2(s[e] * row_lane<e>(vs[grp]), s[e + 1] * row_lane<e + 1>(vs[grp]));
                });
#pragma unroll
                for (int g = grp * PER; g < (grp + 1) * PER; ++g)
                    o[g] = __builtin_amdgcn_mfma_f32_32x32x16_f16(
                        __builtin_bit_cast(h8, vt[buf][32 * g + r32][4 * x + 2 * m2 + h]), __builtin_bit_cast(h8, y), o[g], 0, 0, 0);
            });
        });
    };

    const auto compute = [&](int step, auto bc) {
        constexpr int buf = decltype(bc)::value;
        const int t0 = step * kKeys;
        if (t0 >= hi_any || t0 + (kKeys - 1) < lo_any)
            return;
        float ks[2][NG], vs[2][NG];
        uint32_t big = 0;
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                ks[x][g] = ksc[buf][g][32 * x + lane_key];
                vs[x][g] = vsc[buf][g][32 * x + lane_key];
                big = max(big, __float_as_uint(vs[x][g]));   // a sign counts as not finite: it is looked at
            }
        const bool some_hidden = t0 < lo_all || t0 + kKeys > hi_all || __ballot(not_there(ks[0][0]) || not_there(ks[1][0]));
        if (__ballot(big >= scale_cap)) {                // rare: values larger than any before
            big = max_rows_u32(group_max_u32<16>(big));
            if (some_hidden || big >= kNotFinite) {
                // only what a row sees counts for it
                const auto before = [&](int edge, int x) {   // how many of the lane's 16 keys of half x
                    const int u = min(max(edge - t0 - 32 * x - 4 * h, 0), 32);
                    return (u >> 3) * 4 + min(u & 7, 4);
                };
                const int from0 = before(lo, 0), from1 = before(lo, 1), to0 = before(hi, 0), to1 = before(hi, 1);
                const int row16 = lane & 48;
                uint32_t seen[NG] = {};
                if (t0 >= lo_all) {
                    // the rows see the first so many of a half: maxima over as many lanes
                    const int at0 = row16 + max(to0 - 1, 0), at1 = row16 + max(to1 - 1, 0);
#pragma unroll
                    for (int g = 0; g < NG; ++g) {
                        const uint32_t v0 = __shfl(prefix_max16(abs_bits(vs[0][g])), at0);
                        const uint32_t v1 = __shfl(prefix_max16(abs_bits(vs[1][g])), at1);
                        seen[g] = max(to0 ? v0 : 0u, to1 ? v1 : 0u);
                    }
                } else if (!__ballot((from0 > 0 && from0 < to0 && to0 < 16) || (from1 > 0 && from1 < to1 && to1 < 16))) {
                    // or the last so many
                    const int at0 = row16 + (from0 ? from0 & 15 : max(to0 - 1, 0));
                    const int at1 = row16 + (from1 ? from1 & 15 : max(to1 - 1, 0));
#pragma unroll
                    for (int g = 0; g < NG; ++g) {
                        const uint32_t v0 = abs_bits(vs[0][g]), v1 = abs_bits(vs[1][g]);
                        const uint32_t f0 = __shfl(prefix_max16(v0), at0), l0 = __shfl(suffix_max16(v0), at0);
                        const uint32_t f1 = __shfl(prefix_max16(v1), at1), l1 = __shfl(suffix_max16(v1), at1);
                        seen[g] = max(from0 < to0 ? (from0 ? l0 : f0) : 0u, from1 < to1 ? (from1 ? l1 : f1) : 0u);
                    }
                } else {
                    // or some between: each lane's scales go round the 16 lanes
                    const uint32_t sees0 = (1u << to0) - (1u << min(to0, from0));
                    const uint32_t sees1 = (1u << to1) - (1u << min(to1, from1));
                    uint32_t at = lane & 15;
#pragma unroll 1
                    for (int i = 0; i < 16; ++i) {
                        const bool keep0 = sees0 >> at & 1, keep1 = sees1 >> at & 1;
#pragma unroll
                        for (int g = 0; g < NG; ++g) {
                            seen[g] = max(seen[g], keep0 ? abs_bits(vs[0][g]) : 0u);
                            seen[g] = max(seen[g], keep1 ? abs_bits(vs[1][g]) : 0u);
                            vs[0][g] = next_of_16(vs[0][g]);
                            vs[1][g] = next_of_16(vs[1][g]);
                        }
                        at = (at + 1) & 15;
                    }
                }
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    const uint32_t most = max_halves_u32(seen[g]);
                    const bool finite = most < kNotFinite;
                    scale_exp = max(scale_exp, finite ? exponent_of(most) : kNoScale);
                    spoilt |= finite ? 0u : 1u << g;
                }
                // and the weight 0 of an unseen key stays 0
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int g = 0; g < NG; ++g)
                        vs[x][g] = abs_bits(vs[x][g]) >= kNotFinite ? 0.0f : vs[x][g];
                const int least = group_min_exponent<16>(scale_exp);
                scale_cap = cap_of(min(__builtin_amdgcn_readlane(least, 0), __builtin_amdgcn_readlane(least, 16)));
            } else {
                scale_exp = max(scale_exp, exponent_of(big));
                scale_cap = max(scale_cap, cap_of(__builtin_amdgcn_readfirstlane(max(kNoScale, exponent_of(big)))));
            }
            bound = bound_for(ref, scale_exp);
        }
        const float ks0 = ks[0][0], ks1 = ks[1][0];
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int g = 0; g < NG; ++g)
                ks[x][g] *= score_scale;
        const std::integral_constant<int, 0> first_half;
        const std::integral_constant<int, 1> second_half;
        float s0[16], s1[16];
        scores(s0, ks[0], first_half, bc);
        if (some_hidden)
            hide(s0, ks0, t0);
        const float m0 = largest(s0);
        if (__ballot(m0 > bound))                        // rare after the first tiles
            rescale(m0, nullptr, 0);
        // keeps the lane moves of the scales in this block, where they fold into the products
#pragma unroll
        for (int g = 0; g < NG; ++g)
            asm("" : "+v"(ks[1][g]));
        scores(s1, ks[1], second_half, bc);              // beside these keys' products: the first half's weights
        weights(s0);
        if (some_hidden)
            hide(s1, ks1, t0 + 32);
        const float m1 = largest(s1);
        if (__ballot(m1 > bound))
            rescale(m1, s0, 16);
#pragma unroll
        for (int g = 0; g < NG; ++g)
            asm("" : "+v"(vs[0][g]), "+v"(vs[1][g]));
        output(s0, vs[0], first_half, bc);
        weights(s1);
        output(s1, vs[1], second_half, bc);
    };

    if (s0 < s1) {
        pages_of(s0);
        fetch(s0);
        pages_of(s0 + 1);
    }
    const auto one = [&](int step, auto bc) {
        produce(bc);
        if (step + 1 < s1) {
            fetch(step + 1);
            pages_of(step + 2);
        }
        lds_barrier();
        compute(step, bc);
    };
    // in pairs: the buffers' addresses are constants of the instructions
    for (int step = s0; step < s1; step += 2) {
        one(step, std::integral_constant<int, 0>());
        if (step + 1 < s1)
            one(step + 1, std::integral_constant<int, 1>());
    }

    if (spoilt) {
#pragma unroll
        for (int g = 0; g < N32; ++g)
#pragma unroll
            for (int e = 0; e < 16; ++e)
                o[g][e] = spoilt >> (g / PER) & 1 ? NAN : o[g][e];
    }
    l = sum_halves(l);
    if (parts > 1) {
        // ---- parts: left in the workspace in the order of the registers (a wave's
        // lanes side by side); the last to arrive takes all up again, in order
        const auto slot_of = [&](int p) { return w.base + (int64_t)(slot0 + p) * w.slot_rows * (D + 2); };
        const int at_o = wave * (N32 * 1024) + lane * 2, at_l = kRows * D + (32 * wave + r32) * 2;
        constexpr int AT_ONCE = D < 256 ? 2 : 1;         // parts whose loads are in flight
        float *mine = slot_of(part - part0);
#pragma unroll
        for (int g = 0; g < N32; ++g)
#pragma unroll
            for (int e = 0; e < 16; e += 2)
                store_shared(mine + at_o + g * 1024 + e * 64, o[g][e], o[g][e + 1]);
        if (h == 0)
            store_shared(mine + at_l, l != 0.0f ? ref : -INFINITY, l);
        __builtin_amdgcn_s_waitcnt(0);                   // this wave's stores are complete
        __syncthreads();
        if (threadIdx.x == 0)
            last = arrive(counter, parts) ? 1 : 0;
        __syncthreads();
        if (!last)
            return;
        ref = -INFINITY;
        l = 0.0f;
        for (int p = 0; p < parts; p += AT_ONCE) {
            float2 rl[AT_ONCE], x[AT_ONCE][N32 * 8];
#pragma unroll
            for (int y = 0; y < AT_ONCE; ++y) {
                rl[y] = make_float2(-INFINITY, 0.0f);
                if (p + y < parts) {
                    const float *src = slot_of(p + y);
                    rl[y] = load_shared(src + at_l);
#pragma unroll
                    for (int i = 0; i < N32 * 8; ++i)
                        x[y][i] = load_shared(src + at_o + i * 128);
                }
            }
#pragma unroll
            for (int y = 0; y < AT_ONCE; ++y) {
                if (p + y >= parts)
                    break;
                const float nref = fmaxf(ref, rl[y].y != 0.0f ? rl[y].x : -INFINITY);
                const float f0 = ref == -INFINITY ? 0.0f : exp2_hw(ref - nref);
                const float f1 = rl[y].y != 0.0f ? exp2_hw(rl[y].x - nref) : 0.0f;
                l = l * f0 + rl[y].y * f1;
                ref = nref;
#pragma unroll
                for (int g = 0; g < N32; ++g)
#pragma unroll
                    for (int e = 0; e < 16; e += 2) {
                        const float2 v = x[y][g * 8 + e / 2];
                        o[g][e] = fmaf(v.x, f1, p + y ? o[g][e] * f0 : 0.0f);
                        o[g][e + 1] = fmaf(v.y, f1, p + y ? o[g][e + 1] * f0 : 0.0f);
                    }
            }
        }
    }

    // ---- results: the lane's row, dims 32 g + 8 i + 4 h ..+3
    if (row < rows) {
        const float inv = l != 0.0f ? 1.0f / l : 0.0f;
        const int64_t at = (int64_t)(seq.q0 + qi) * a.q_heads + head * group + hh;
#pragma unroll
        for (int g = 0; g < N32; ++g)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                *reinterpret_cast<uint2 *>(a.out + at * D + 32 * g + 8 * i + 4 * h) =
                    make_uint2(pack_h2(o[g][4 * i] * inv, o[g][4 * i + 1] * inv), pack_h2(o[g][4 * i + 2] * inv, o[g][4 * i + 3] * inv));
        if (a.lse && h == 0)
            a.lse[at] = l != 0.0f ? (ref + __builtin_amdgcn_logf(l)) * kLn2 : -INFINITY;
    }
}

}  // namespace

void launch_kv4_prefill(const Kv4Cache &c, const Kv4AttnArgs &a, int row_limit, void *workspace, hipStream_t st)
{
    const Kv4Tiles t = kv4_prefill_tiles(a.T, a.B, a.group, c.heads, (int64_t)a.max_pages << c.shift);
    Partial w;
    w.grid = (int)t.grid;
    w.row_limit = row_limit;
    w.slot_rows = kRows;
    w.slots = (int)t.slots;
    w.over_group = over_group(a.group);
    w.counters = static_cast<uint64_t *>(workspace);
    w.base = reinterpret_cast<float *>(static_cast<char *>(workspace) + kv4_counter_bytes(t.slots, 1));
    const dim3 grid((unsigned)t.grid), block(kThreads);
    const auto launch = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, block, 0, st, c, a, w); };
    switch (c.D * 8 + c.D / c.G) {
    case 64 * 8 + 1: launch(kv4_prefill_kernel<64, 1>); return;
    case 64 * 8 + 2: launch(kv4_prefill_kernel<64, 2>); return;
    case 128 * 8 + 1: launch(kv4_prefill_kernel<128, 1>); return;
    case 128 * 8 + 2: launch(kv4_prefill_kernel<128, 2>); return;
    case 128 * 8 + 4: launch(kv4_prefill_kernel<128, 4>); return;
    case 256 * 8 + 1: launch(kv4_prefill_kernel<256, 1>); return;
    case 256 * 8 + 2: launch(kv4_prefill_kernel<256, 2>); return;
    default: launch(kv4_prefill_kernel<256, 4>); return;
    }
}

}  // namespace w4a8

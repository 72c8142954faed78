// Attention of few query rows over the 4-bit cache (include/w4a8.h:
// kv4_attention): up to 32 rows (queries x query heads of a kv head) a sequence
// and kv head, so that the cache is read once.
//
// What bounds it: for long caches reading it, D + 8 D / G bytes for a key and
// value of one head; for short ones the chain of loads, steps and joins.
// Measured: one sequence of 131075 keys (151 MB) 39.5 us, 3.8 TB/s over the whole
// call; 32 sequences of up to 4516 (81.5 MB) 23.4 us; one of 517 9.7 us.  About
// 60 % of a workgroup's cycles are steps in the first, 40 % in the second.
//
// One wavefront takes steps of 32 keys.  S^T =
// K Q^T on 16x16x32 matrix instructions with the codes as fp16 (exact) and the
// keys' scales applied to the fp32 scores; the result leaves a lane with one
// query row and four consecutive keys of each 16, which is, for two pieces of
// 16, the operand of the second product O^T = V^T P^T as it stands.  The
// cache's byte order gives a lane its operand bytes side by side: K's as one
// load of D / 8 bytes, V's as D / 32 bytes of each of its keys.  The loads of
// the next steps are in flight while one is computed.
//
// The keys of a (sequence, head) are cut into parts of at most `limit` steps,
// the same limit for all, so that a workgroup (four waves, joined in LDS) has
// one part whatever the sequences' lengths; a workgroup finds its own from a
// scan of the lengths.  Where there are several parts each is left in the
// workspace and the last to arrive joins them in order, so the result does
// not depend on who that is.
#include "kv4_device.hpp"
#include "lds_copy.hpp"

namespace w4a8 {

namespace {


constexpr int kWaves = 4, kThreads = 64 * kWaves;

// What a lane loads for a step of P pieces of 16 keys.  Of the scales, which
// the 16 lanes of a row share, a lane takes one key's of every second piece:
// lane 8 x + 4 v + j of a row K's (v = 0) or V's (v = 1) of key
// 4 (lane / 16) + j of the pieces 2 h + x.
template <int P, int N32, int NG> struct Step {
    uint32_t k[P][N32];                 // key lane % 16: dims 32 i + 8 (lane / 16) ..+7
    uint32_t v[P][4][(N32 + 3) / 4];    // keys 4 (lane / 16) + j: dims 32 g + 2 (lane % 16) ..+1
    float sc[P / 2][NG];
    uint32_t ok;                        // bit p: the page of piece p exists
};

// A lane's offsets into a piece's rows.
struct LaneAt {
    uint32_t k, v;              // bytes
    int64_t scale;              // bytes from K's scales of the piece
    bool odd;                   // scales of the odd pieces
};

template <int P, int D, int NG>
__device__ __forceinline__ void load_step(Step<P, D / 32, NG> &s, const Kv4Cache &c, int head, const int (&page)[P],
                                          int step, const LaneAt &at)
{
    constexpr int N32 = D / 32;
    const char *scales = nullptr;
    s.ok = 0;
#pragma unroll
    for (int p = 0; p < P; ++p) {
        const bool ok = kv4_page_ok(page[p], c.pages);
        s.ok |= ok ? 1u << p : 0u;
        const int64_t row = c.row(ok ? page[p] : 0, head, (step * (16 * P) + p * 16) & ((1 << c.shift) - 1));
        const uint8_t *kp = c.k + row * (D / 2), *vp = c.v + row * (D / 2);
        const char *sr = reinterpret_cast<const char *>(c.ks + row * NG);
        scales = p % 2 && !at.odd ? scales : sr;
        if constexpr (N32 == 2) {
            const uint2 w = *reinterpret_cast<const uint2 *>(kp + at.k);
            s.k[p][0] = w.x, s.k[p][1] = w.y;
        } else {
#pragma unroll
            for (int i = 0; i < N32 / 4; ++i) {
                const v4u w = *reinterpret_cast<const v4u *>(kp + (at.k + 16 * i));
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    s.k[p][4 * i + e] = w[e];
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint8_t *q = vp + (at.v + j * (D / 2));
            if constexpr (N32 == 2) {
                s.v[p][j][0] = *reinterpret_cast<const uint16_t *>(q);
            } else if constexpr (N32 == 4) {
                s.v[p][j][0] = *reinterpret_cast<const uint32_t *>(q);
            } else {
                const uint2 w = *reinterpret_cast<const uint2 *>(q);
                s.v[p][j][0] = w.x, s.v[p][j][1] = w.y;
            }
        }
        if (p % 2 == 0)
            continue;
        const float *sp = reinterpret_cast<const float *>(scales + at.scale);
        if constexpr (NG == 1) {
            s.sc[p / 2][0] = *sp;
        } else if constexpr (NG == 2) {
            const float2 w = *reinterpret_cast<const float2 *>(sp);
            s.sc[p / 2][0] = w.x, s.sc[p / 2][1] = w.y;
        } else {
            const v4f w = *reinterpret_cast<const v4f *>(sp);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                s.sc[p / 2][e] = w[e];
        }
    }
}

// A row's output and log of the softmax sum from its joined part.  Here and
// below a sum of 0 is a row that sees nothing; one that is no number stays so.
template <int D>
__device__ __forceinline__ void store_row(const Partial &w, const Kv4AttnArgs &a, const Kv4Seq &seq, int head, int row,
                                          int d, float4 sum, float ref, float l)
{
    const float inv = l != 0.0f ? 1.0f / l : 0.0f;
    const int i = query_of(row, w.over_group, a.group);
    const int64_t at = (int64_t)(seq.q0 + i) * a.q_heads + head * a.group + (row - i * a.group);
    *reinterpret_cast<uint2 *>(a.out + at * D + d) =
        make_uint2(pack_h2(sum.x * inv, sum.y * inv), pack_h2(sum.z * inv, sum.w * inv));
    if (a.lse && d == 0)
        a.lse[at] = l != 0.0f ? (ref + __builtin_amdgcn_logf(l)) * kLn2 : -INFINITY;
}

// Joins the parts in `parts` slots from slot p0 on: `rows` rows of their
// (sequence, head).  A thread takes four dims of a row; where there are more threads, groups of them take every
// so-many-th part and are joined in LDS.  Parts come from memory at some
// microseconds' latency, so eight are in flight at a time.
template <int D>
__device__ void join_parts(const Partial &w, const Kv4AttnArgs &a, const Kv4Seq &seq, int head, int rows, int p0,
                           int parts, float *lds)
{
    const int p1 = p0 + parts - 1;
    constexpr int kAhead = 8;
    const int items = rows * (D / 4);
    const int groups = items < kThreads ? kThreads / items : 1;
    const int grp = items < kThreads ? threadIdx.x / items : 0;
    for (int x0 = 0; x0 < items; x0 += kThreads) {
        const int x = x0 + (items < kThreads ? threadIdx.x - grp * items : threadIdx.x);
        const int row = x / (D / 4), d = x % (D / 4) * 4;
        float R = -INFINITY, L = 0.0f;
        float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (x < items && grp < groups) {
            for (int p = p0 + grp; p <= p1; p += groups * kAhead) {
                float2 rl[kAhead], u[kAhead], v[kAhead];
#pragma unroll
                for (int i = 0; i < kAhead; ++i) {
                    rl[i] = u[i] = v[i] = make_float2(0.0f, 0.0f);
                    const int pp = p + i * groups;
                    if (pp <= p1) {                      // each load goes to memory: none for nothing
                        const float *src = w.base + ((int64_t)pp * w.slot_rows + row) * (D + 2);
                        rl[i] = load_shared(src + D);
                        u[i] = load_shared(src + d);
                        v[i] = load_shared(src + d + 2);
                    }
                }
                float top = R;
#pragma unroll
                for (int i = 0; i < kAhead; ++i)
                    top = fmaxf(top, rl[i].y != 0.0f ? rl[i].x : -INFINITY);
                const float keep = R == -INFINITY ? 0.0f : exp2_hw(R - top);
                L *= keep;
                sum.x *= keep, sum.y *= keep, sum.z *= keep, sum.w *= keep;
#pragma unroll
                for (int i = 0; i < kAhead; ++i) {
                    const float f = rl[i].y != 0.0f ? exp2_hw(rl[i].x - top) : 0.0f;
                    L = fmaf(rl[i].y, f, L);
                    sum.x = fmaf(u[i].x, f, sum.x), sum.y = fmaf(u[i].y, f, sum.y);
                    sum.z = fmaf(v[i].x, f, sum.z), sum.w = fmaf(v[i].y, f, sum.w);
                }
                R = top;
            }
        }
        if (groups > 1) {
            float *mine = lds + threadIdx.x * 6;
            mine[0] = R, mine[1] = L, mine[2] = sum.x, mine[3] = sum.y, mine[4] = sum.z, mine[5] = sum.w;
            __syncthreads();
            if (grp == 0 && x < items) {
                for (int g = 1; g < groups; ++g) {
                    const float *o = lds + (g * items + x) * 6;
                    const float top = fmaxf(R, o[0]);
                    const float f0 = R == -INFINITY ? 0.0f : exp2_hw(R - top);
                    const float f1 = o[0] == -INFINITY ? 0.0f : exp2_hw(o[0] - top);
                    R = top;
                    L = L * f0 + o[1] * f1;
                    sum.x = sum.x * f0 + o[2] * f1, sum.y = sum.y * f0 + o[3] * f1;
                    sum.z = sum.z * f0 + o[4] * f1, sum.w = sum.w * f0 + o[5] * f1;
                }
            }
        }
        if (grp == 0 && x < items)
            store_row<D>(w, a, seq, head, row, d, sum, R, L);
    }
}

template <int D, int NG, int RT>
__global__ __launch_bounds__(kThreads, RT * D == 512 ? 1 : 2) void kv4_decode_kernel(Kv4Cache c, Kv4AttnArgs a,
                                                                                                 Partial w)
{
    constexpr int N32 = D / 32, PER = N32 / NG;          // steps of 32 dims, of one group
    constexpr int P = 2, KEYS = 16 * P;                  // pieces of 16 keys and keys of a step
    constexpr int LD = D + 4;                            // LDS row: 16 rows of float4 without bank conflicts
    __shared__ float os[kWaves][16][LD];
    __shared__ float refs[kWaves][16 * RT], ls[kWaves][16 * RT];
    __shared__ int last;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, b4 = lane >> 4;
    const int group = a.group, B = a.B;

    // ---- this workgroup's part: sequences 64 at a time, one a lane
    Kv4Seq sl;                                           // sequence base + lane
    int nl;                                              // and its steps
    const auto lookup = [&](int base) {
        nl = 0;
        if (base + lane < B) {
            sl = kv4_sequence(a, c.shift, base + lane);
            if ((int64_t)sl.m * group <= w.row_limit)
                nl = kv4_steps(sl, a.causal, a.window, KEYS).count;
        }
    };
    int64_t steps = 0;                                   // of all sequences
    int longest = 0;                                     // of one
    for (int base = 0; base < B; base += 64) {
        lookup(base);
        steps += group_sum_u32<64>((uint32_t)nl);
        longest = max(longest, (int)group_max_u32<64>((uint32_t)nl));
    }
    const int limit = kv4_part_limit(steps * c.heads, longest, KEYS);
    int b = -1, count = 0, parts = 0, id = blockIdx.x;   // id: within the sequences from b on
    Kv4Seq seq = {0, 0, 0, 0};
    for (int base = 0; base < B; base += 64) {
        if (B > 64)
            lookup(base);
        const int k = (nl + limit - 1) / limit;
        const int inc = prefix_sum(k * c.heads);
        const uint64_t past = __ballot(inc > id);
        if (past) {
            const int at = __builtin_ctzll(past);
            b = base + at;
            count = __builtin_amdgcn_readlane(nl, at);
            parts = __builtin_amdgcn_readlane(k, at);
            seq.q0 = __builtin_amdgcn_readlane(sl.q0, at);
            seq.m = __builtin_amdgcn_readlane(sl.m, at);
            seq.n = __builtin_amdgcn_readlane(sl.n, at);
            seq.rest = __builtin_amdgcn_readlane(sl.rest, at);
            id -= __builtin_amdgcn_readlane(inc, at) - parts * c.heads;
            break;
        }
        id -= __builtin_amdgcn_readlane(inc, 63);
    }
    if (b < 0)
        return;
    const int head = (uint32_t)id / (uint32_t)parts, part = id - head * parts;
    const int rows = seq.m * group;
    const int first = kv4_steps(seq, a.causal, a.window, KEYS).first;
    const int64_t item = (int64_t)b * c.heads + head;
    if (parts > 1 && threadIdx.x == 0)
        announce(w.counters + item * kCounterStride, a.tag);

    // ---- this wave's steps (none where there are no keys) and its first loads
    const int s0 = kv4_split(count, parts, part), s1 = kv4_split(count, parts, part + 1);
    const int n = seq.n > 0 ? s1 - s0 : 0;
    const int w0 = first + s0 + n * wave / kWaves, w1 = first + s0 + n * (wave + 1) / kWaves;
    const int32_t *table = a.table + (int64_t)b * a.max_pages;
    const int last_piece = (seq.n - 1) >> 4;
    // the pages of a step's pieces of 16 keys (behind the last key the last page, where nothing is seen)
    int page[P];
    const auto pages_of = [&](int step) {
#pragma unroll
        for (int p = 0; p < P; ++p)
            page[p] = scalar_load(table + ((int64_t)min(step * P + p, last_piece) * 16 >> c.shift));
    };
    LaneAt at;
    at.k = r * (D / 2) + b4 * (D / 8);
    at.v = 4 * b4 * (D / 2) + r * N32;
    at.odd = (r & 8) != 0;
    at.scale = ((r & 4) ? reinterpret_cast<const char *>(c.vs) - reinterpret_cast<const char *>(c.ks) : 0) +
               (4 * b4 + (r & 3)) * NG * 4;
    const auto fetch = [&](Step<P, N32, NG> &s, int step) { load_step<P, D, NG>(s, c, head, page, step, at); };
    Step<P, N32, NG> next;
    if (w0 < w1) {
        pages_of(w0);
        fetch(next, w0);
        pages_of(w0 + 1);
    }

    // ---- queries: row lane % 16 of each 16, visible keys [lo, hi)
    h8 q[RT][N32];
    int lo[RT], hi[RT];
    float ref[RT], bound[RT], l[RT];
    v4f o[RT][2 * N32];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        const int row = 16 * t + r;
        const int rc = row < rows ? row : rows - 1;      // rows past the last repeat it and are not stored
        const int i = query_of(rc, w.over_group, group), hh = rc - i * group;
        const uint16_t *qp = a.q + (int64_t)(seq.q0 + i) * a.q_stride + (int64_t)(head * group + hh) * D + 8 * b4;
#pragma unroll
        for (int k = 0; k < N32; ++k)
            q[t][k] = order8(*reinterpret_cast<const uint4 *>(qp + 32 * k));
        lo[t] = kv4_lo(seq, i, a.window);
        hi[t] = kv4_hi(seq, i, a.causal);
        ref[t] = bound[t] = kFarBelow;
        l[t] = 0.0f;
#pragma unroll
        for (int k = 0; k < 2 * N32; ++k)
            o[t][k] = (v4f){0.0f, 0.0f, 0.0f, 0.0f};
    }
    const int lo_most = kv4_lo(seq, seq.m - 1, a.window), hi_least = kv4_hi(seq, 0, a.causal);
    const int lo_first = kv4_lo(seq, 0, a.window), hi_last = kv4_hi(seq, seq.m - 1, a.causal);
    // exponent of the largest value scale that a row has seen; bits of 2^(e + 1)
    // for the smallest of them
    int scale_exp[RT];
    uint32_t scale_cap = 0;
    uint32_t spoilt[RT];                                 // bit g: it has seen one of group g that is not finite
#pragma unroll
    for (int t = 0; t < RT; ++t)
        scale_exp[t] = kNoScale, spoilt[t] = 0;
    const float score_scale = a.scale * kLog2e;
    // Where a row sees few keys, one rounding of a weight is in every element of
    // its output: the weights are taken as two fp16 values, 22 bits, if any row
    // of the sequence sees so few.  (With more keys the roundings average out and
    // the second product costs 6 to 9 %.)
    const bool fine = hi_least - lo_first <= kFewKeys;

    const auto compute = [&](const Step<P, N32, NG> &cur, int step) {
        const int t0 = step * KEYS;
        float sc[P / 2][NG], ksc[P / 2][NG];
#pragma unroll
        for (int h = 0; h < P / 2; ++h)
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                sc[h][g] = cur.sc[h][g];
                ksc[h][g] = cur.sc[h][g] * score_scale;
            }
        // scores
        float s[RT][P][4];
        each<P>([&](auto pc) {
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
                    const float f = row_lane<8 * (p % 2) + j>(ksc[p / 2][g]);
#pragma unroll
                    for (int t = 0; t < RT; ++t)
                        s[t][p][j] = g == 0 ? acc[t][j] * f : fmaf(acc[t][j], f, s[t][p][j]);
                });
            });
        });
        // a step that not every row sees whole: hide keys, whatever stands for them
        uint32_t some_hidden = 0;                        // a number: branching on the condition twice cost 17 registers
        if (cur.ok != (1u << P) - 1 || t0 < lo_most || t0 > hi_least - KEYS) {
            some_hidden = seq.m > 1 ? kNotFinite : 0u;   // one query's rows all see the same
#pragma unroll
            for (int p = 0; p < P; ++p) {
                const bool there = (cur.ok >> p) & 1;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int key = t0 + 16 * p + 4 * b4 + j;
#pragma unroll
                    for (int t = 0; t < RT; ++t)
                        s[t][p][j] = there && key >= lo[t] && key < hi[t] ? s[t][p][j] : -INFINITY;
                }
            }
            // values that no row sees
#pragma unroll
            for (int h = 0; h < P / 2; ++h) {
                const int mine = t0 + 32 * h + 2 * (r & 8) + 4 * b4 + (r & 3);
                const bool there = (cur.ok >> (2 * h + (r >> 3)) & 1) && mine >= lo_first && mine < hi_last;
#pragma unroll
                for (int g = 0; g < NG; ++g)
                    sc[h][g] = there ? sc[h][g] : 0.0f;
            }
        }
        uint32_t big = 0;                                // of the value scales
#pragma unroll
        for (int h = 0; h < P / 2; ++h)
#pragma unroll
            for (int g = 0; g < NG; ++g)
                big = max(big, abs_bits(sc[h][g]));
        big = (r & 4) ? big : 0u;
        if (__ballot(big >= scale_cap)) {                // rare: values larger than any before
            big = max_rows_u32(group_max_u32<16>(big)) | some_hidden;
            if (__builtin_amdgcn_readfirstlane(big) >= kNotFinite) {
                // only what a row sees counts for it (a hidden key's score is -infinity)
                uint32_t seen[RT][NG] = {};
                each<4 * P>([&](auto ic) {
                    constexpr int p = decltype(ic)::value / 4, j = decltype(ic)::value % 4;
                    uint32_t keep[RT];
#pragma unroll
                    for (int t = 0; t < RT; ++t)
                        keep[t] = s[t][p][j] != -INFINITY ? 0x7fffffffu : 0u;
                    each<NG>([&](auto gc) {
                        constexpr int g = decltype(gc)::value;
                        const uint32_t v = __float_as_uint(row_lane<8 * (p % 2) + 4 + j>(sc[p / 2][g]));
#pragma unroll
                        for (int t = 0; t < RT; ++t)
                            seen[t][g] = max(seen[t][g], v & keep[t]);
                    });
                });
#pragma unroll
                for (int t = 0; t < RT; ++t)
#pragma unroll
                    for (int g = 0; g < NG; ++g) {
                        const uint32_t most = max_rows_u32(seen[t][g]);
                        const bool finite = most < kNotFinite;
                        scale_exp[t] = max(scale_exp[t], finite ? exponent_of(most) : kNoScale);
                        spoilt[t] |= finite ? 0u : 1u << g;
                    }
                // and the weight 0 of an unseen key stays 0
#pragma unroll
                for (int h = 0; h < P / 2; ++h)
#pragma unroll
                    for (int g = 0; g < NG; ++g)
                        sc[h][g] = abs_bits(sc[h][g]) >= kNotFinite ? 0.0f : sc[h][g];
                int least = scale_exp[0];
#pragma unroll
                for (int t = 1; t < RT; ++t)
                    least = min(least, scale_exp[t]);
                scale_cap = cap_of(__builtin_amdgcn_readfirstlane(group_min_exponent<16>(least)));
            } else {
#pragma unroll
                for (int t = 0; t < RT; ++t)
                    scale_exp[t] = max(scale_exp[t], exponent_of(big));
                scale_cap = max(scale_cap, cap_of(__builtin_amdgcn_readfirstlane(max(kNoScale, exponent_of(big)))));
            }
#pragma unroll
            for (int t = 0; t < RT; ++t)
                bound[t] = bound_for(ref[t], scale_exp[t]);
        }
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            float m = max3(s[t][0][0], s[t][0][1], s[t][0][2]);
            m = max3(m, s[t][0][3], s[t][1][0]);
            m = max3(m, s[t][1][1], s[t][1][2]);
            m = max3(m, s[t][1][3], s[t][1][3]);
            if (__ballot(m > bound[t])) {                // rare after the first steps
                m = max_rows(m, m);
                if (m > bound[t]) {
                    const float nref = reference_for(ref[t], m, scale_exp[t]);
                    const float alpha = exp2_hw(ref[t] - nref);   // 0 before the first key
                    l[t] *= alpha;
                    ref[t] = nref;
                    bound[t] = bound_for(nref, scale_exp[t]);
#pragma unroll
                    for (int k = 0; k < 2 * N32; ++k)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            o[t][k][e] *= alpha;
                }
            }
#pragma unroll
            for (int p = 0; p < P; ++p) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    s[t][p][j] = exp2_hw(s[t][p][j] - ref[t]);
                l[t] += (s[t][p][0] + s[t][p][1]) + (s[t][p][2] + s[t][p][3]);
            }
        }
        // weights times the values' scales, rounded to fp16; what is left of them after that
        const auto weights = [&](h8 (&wt)[RT][P / 2][NG], bool rest) {
#pragma unroll
            for (int t = 0; t < RT; ++t)
                each<P / 2>([&](auto hc) {
                    constexpr int h = decltype(hc)::value;
                    each<NG>([&](auto gc) {
                        constexpr int g = decltype(gc)::value;
                        u32x4 x;
                        each<4>([&](auto ic) {
                            constexpr int x2 = decltype(ic)::value / 2, j = decltype(ic)::value % 2 * 2;
                            const float a0 = s[t][2 * h + x2][j] * row_lane<8 * x2 + 4 + j>(sc[h][g]);
                            const float a1 = s[t][2 * h + x2][j + 1] * row_lane<8 * x2 + 5 + j>(sc[h][g]);
                            const uint32_t top = pack_h2(a0, a1);
                            x[decltype(ic)::value] = rest ? pack_h2(a0 - lo_h2f(top), a1 - hi_h2f(top)) : top;
                        });
                        wt[t][h][g] = __builtin_bit_cast(h8, x);
                    });
                });
        };
        // O^T += V^T P^T: 16 rows 32 g + 2 r + e of the values for byte g's two nibbles e
        const auto output = [&](const h8 (&wt)[RT][P / 2][NG]) {
            each<P / 2>([&](auto hc) {
                constexpr int h = decltype(hc)::value;
                each<N32>([&](auto gc) {
                    constexpr int g = decltype(gc)::value;
                    const auto &p0 = cur.v[2 * h], &p1 = cur.v[2 * h + 1];
                    const uint32_t x0 = byte_pair<g % 4>(p0[0][g / 4], p0[1][g / 4]), x1 = byte_pair<g % 4>(p0[2][g / 4], p0[3][g / 4]);
                    const uint32_t x2 = byte_pair<g % 4>(p1[0][g / 4], p1[1][g / 4]), x3 = byte_pair<g % 4>(p1[2][g / 4], p1[3][g / 4]);
                    const u32x4 e0 = {codes_low(x0), codes_low(x1), codes_low(x2), codes_low(x3)};
                    const u32x4 e1 = {codes_high(x0), codes_high(x1), codes_high(x2), codes_high(x3)};
#pragma unroll
                    for (int t = 0; t < RT; ++t) {
                        const h8 x = wt[t][h][g / PER];
                        o[t][2 * g] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, e0), x, o[t][2 * g], 0, 0, 0);
                        o[t][2 * g + 1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, e1), x, o[t][2 * g + 1], 0, 0, 0);
                    }
                });
            });
        };
        h8 wt[RT][P / 2][NG];
        weights(wt, false);
        output(wt);
        if (fine) {
            weights(wt, true);
            output(wt);
        }
    };
    // The next step's loads are in flight during one, its pages (scalar loads)
    // are a step further ahead; other waves hide the rest.  The step stands in
    // the code once: a short call is bound by fetching instructions, and with
    // two steps ahead in five copies it took as long.
    for (int step = w0; step < w1; ++step) {
        const Step<P, N32, NG> cur = next;
        if (step + 1 < w1) {
            fetch(next, step + 1);
            pages_of(step + 2);
        }
        compute(cur, step);
    }

    // ---- join the four waves
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        l[t] = sum_rows(l[t]);
        if (lane < 16) {
            refs[wave][16 * t + r] = l[t] != 0.0f ? ref[t] : -INFINITY;
            ls[wave][16 * t + r] = l[t];
        }
    }
    lds_barrier();
    float *slot = w.base + (int64_t)blockIdx.x * w.slot_rows * (D + 2);
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        if (16 * t >= rows)
            break;
        if (16 * t + r < rows) {
            float R = -INFINITY;
#pragma unroll
            for (int x = 0; x < kWaves; ++x)
                R = fmaxf(R, refs[x][16 * t + r]);
            const float keep = l[t] != 0.0f ? exp2_hw(ref[t] - R) : 0.0f;
#pragma unroll
            for (int g = 0; g < N32; ++g) {
                const float f = spoilt[t] >> (g / PER) & 1 ? NAN : keep;
                // lane: dims 32 g + 8 b4 + 2 reg + e
                float4 *dst = reinterpret_cast<float4 *>(&os[wave][r][32 * g + 8 * b4]);
                dst[0] = make_float4(o[t][2 * g][0] * f, o[t][2 * g + 1][0] * f, o[t][2 * g][1] * f, o[t][2 * g + 1][1] * f);
                dst[1] = make_float4(o[t][2 * g][2] * f, o[t][2 * g + 1][2] * f, o[t][2 * g][3] * f, o[t][2 * g + 1][3] * f);
            }
        }
        lds_barrier();
        // a thread: four dims of a row at a time
        const int items = (rows - 16 * t < 16 ? rows - 16 * t : 16) * (D / 4);
        for (int x = threadIdx.x; x < items; x += kThreads) {
            const int rr = x / (D / 4), d = x % (D / 4) * 4, row = 16 * t + rr;
            float RR = -INFINITY, L = 0.0f;
#pragma unroll
            for (int y = 0; y < kWaves; ++y)
                RR = fmaxf(RR, refs[y][row]);
#pragma unroll
            for (int y = 0; y < kWaves; ++y)
                L += ls[y][row] != 0.0f ? ls[y][row] * exp2_hw(refs[y][row] - RR) : 0.0f;
            float4 sum = *reinterpret_cast<const float4 *>(&os[0][rr][d]);
#pragma unroll
            for (int y = 1; y < kWaves; ++y) {
                const float4 v = *reinterpret_cast<const float4 *>(&os[y][rr][d]);
                sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
            }
            if (parts == 1) {
                store_row<D>(w, a, seq, head, row, d, sum, RR, L);
            } else {
                float *dst = slot + row * (D + 2);
                store_shared(dst + d, sum.x, sum.y);
                store_shared(dst + d + 2, sum.z, sum.w);
                if (d == 0)
                    store_shared(dst + D, RR, L);
            }
        }
        if (RT > 1)
            lds_barrier();
    }
    if (parts > 1) {
        // ---- join the workgroups: the last to arrive reads all parts in order
        __builtin_amdgcn_s_waitcnt(0);                   // this wave's stores are complete
        __syncthreads();
        if (threadIdx.x == 0)
            last = arrive(w.counters + item * kCounterStride, parts) ? 1 : 0;
        __syncthreads();
        if (last)
            join_parts<D>(w, a, seq, head, rows, blockIdx.x - part, parts, &os[0][0][0]);
    }
}

template <int D, int NG>
void launch(const Kv4Cache &c, const Kv4AttnArgs &a, const Partial &w, int rows, hipStream_t st)
{
    const dim3 grid((unsigned)w.grid), block(kThreads);
    if (rows <= 16)
        hipLaunchKernelGGL((kv4_decode_kernel<D, NG, 1>), grid, block, 0, st, c, a, w);
    else
        hipLaunchKernelGGL((kv4_decode_kernel<D, NG, 2>), grid, block, 0, st, c, a, w);
}

}  // namespace

void launch_kv4_decode(const Kv4Cache &c, const Kv4AttnArgs &a, int rows, hipStream_t st)
{
    Partial w;
    w.grid = (int)kv4_decode_grid(a.B, c.heads, (int64_t)a.max_pages << c.shift);
    w.row_limit = rows;
    w.slots = w.grid;
    w.slot_rows = rows;
    w.over_group = over_group(a.group);
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

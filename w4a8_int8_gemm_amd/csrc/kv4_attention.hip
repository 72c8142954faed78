// Attention over the 4-bit paged cache (include/w4a8.h: kv4_attention): which
// kernel takes which sequences, and the workspace they share.
#include "kv4.hpp"

namespace w4a8 {

namespace {

// Rows a kv head that the kernel for few rows is launched for: what a sequence
// can have, or that kernel's limit.
int decode_rows(int group, int64_t max_q)
{
    return group * max_q < kDecodeRows ? (int)(group * max_q) : kDecodeRows;
}

size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

size_t decode_bytes(int q_heads, int kv_heads, int D, int64_t T, int B, int max_q)
{
    const int rows = decode_rows(q_heads / kv_heads, max_q < T ? max_q : T);
    return kv4_counter_bytes(B, kv_heads) +
           align256((size_t)(B * (int64_t)kv_heads + kPartsMore) * rows * (D + 2) * sizeof(float));
}

}  // namespace

size_t kv4_attention_workspace(int q_heads, int kv_heads, int D, int64_t T, int B, int max_q)
{
    const int group = q_heads / kv_heads;
    size_t bytes = decode_bytes(q_heads, kv_heads, D, T, B, max_q);
    if ((int64_t)group * (max_q < T ? max_q : T) > kDecodeRows) {
        // any length of keys: the table's width is not known here
        const Kv4Tiles t = kv4_prefill_tiles(T, B, group, kv_heads, int64_t(1) << 30);
        bytes += kv4_counter_bytes(t.slots, 1) + (size_t)t.slots * kTileRows * (D + 2) * sizeof(float);
    }
    return bytes;
}

namespace {

struct Launches {
    bool few, many;
};
Launches launches_of(const Kv4AttnArgs &a)
{
    Launches l;
    l.many = (int64_t)a.group * a.max_q > kDecodeRows;
    // Where one query is too many rows for the kernel for few, or all sequences
    // have max_q queries (they do if T = B max_q and q_starts covers all rows),
    // the other kernel takes them all: one launch instead of two.  It is right
    // for every sequence, so that ranges which cover fewer rows cost time only,
    // and the weights' second part.
    l.few = a.group <= kDecodeRows && !(l.many && a.T == (int64_t)a.B * a.max_q);
    return l;
}

}  // namespace

bool kv4_attention_fits(const Kv4Cache &c, const Kv4AttnArgs &a)
{
    const Launches l = launches_of(a);
    const int64_t most = (int64_t)a.max_pages << c.shift, limit = (int64_t(1) << 24) - 1;
    return (!l.few || kv4_decode_grid(a.B, c.heads, most) <= limit) &&
           (!l.many || kv4_prefill_tiles(a.T, a.B, a.group, c.heads, most).grid <= limit);
}

void launch_kv4_attention(const Kv4Cache &c, const Kv4AttnArgs &a, hipStream_t st)
{
    const Launches l = launches_of(a);
    if (l.few)
        launch_kv4_decode(c, a, decode_rows(a.group, a.max_q), st);
    if (l.many)
        launch_kv4_prefill(c, a, l.few ? kDecodeRows : 0,
                           static_cast<char *>(a.workspace) +
                               decode_bytes(a.group * c.heads, c.heads, c.D, a.T, a.B, a.max_q), st);
}

}  // namespace w4a8

// Integer rules of the attention kernels: what a sequence's entries in the
// device-side tables mean once they are cut to the call's buffers, which keys
// a query sees, and how the work is divided over the workgroups.  Plain C++
// without device code, so that the CPU test suite runs it on hostile tables.
#pragma once

#include <stdint.h>

#if defined(__HIPCC__)
#include <hip/hip_runtime.h>
#define KV4_HD __host__ __device__ __forceinline__
#else
#define KV4_HD static inline
#endif

namespace w4a8 {

// A sequence's queries and keys.
struct Kv4Seq {
    int q0;                     // first query row
    int m;                      // queries, all rows [q0, q0 + m) inside [0, T)
    int n;                      // keys, all inside the table's pages
    int rest;                   // queries past max_q: not computed, but the last of them stands at the last key
};

// From the tables' entries: `start`, `end` the sequence's rows, `len` its keys
// (any values); T rows (< 2^31) in the call, at most max_q of them a sequence's; `most`
// keys in the table's pages (< 2^31).
KV4_HD Kv4Seq kv4_cut(int start, int end, int len, int T, int max_q, int most)
{
    Kv4Seq s;
    s.n = len < 0 ? 0 : len < most ? len : most;
    s.q0 = start < 0 ? 0 : start < T ? start : T;
    end = end < T ? end : T;
    const int all = end > s.q0 ? end - s.q0 : 0;
    s.m = all < max_q ? all : max_q;
    s.rest = all - s.m;
    return s;
}

// The keys [lo, hi) that query i of m sees among n.
KV4_HD int kv4_hi(int n, int m, int i, bool causal)
{
    const int hi = causal ? n - m + i + 1 : n;
    return hi < 0 ? 0 : hi;
}
KV4_HD int kv4_lo(int n, int m, int i, int window)
{
    const int p1 = n - m + i + 1;                       // p1 - window may leave 32 bits where p1 < 0
    return window > 0 && p1 > window ? p1 - window : 0;
}

// Of a sequence's query i.
KV4_HD int kv4_hi(const Kv4Seq &s, int i, bool causal) { return kv4_hi(s.n, s.m + s.rest, i, causal); }
KV4_HD int kv4_lo(const Kv4Seq &s, int i, int window) { return kv4_lo(s.n, s.m + s.rest, i, window); }

// Steps of `keys` keys that a sequence's queries need together; one (empty)
// step where they see nothing, none without queries.
struct Kv4Steps {
    int first, count;
};
KV4_HD Kv4Steps kv4_steps(const Kv4Seq &s, bool causal, int window, int keys)
{
    Kv4Steps r = {0, 0};
    if (s.m == 0)
        return r;
    const int hi = kv4_hi(s, s.m - 1, causal), lo = kv4_lo(s, 0, window);
    r.first = lo / keys;
    r.count = (int)(((int64_t)hi + keys - 1) / keys) - r.first;
    r.count = r.count < 1 ? 1 : r.count;
    return r;
}

// A (sequence, head) of `count` steps is cut into ceil(count / limit) even
// parts.  With the limit below there are at most kPartsMore more of them in
// all than (sequence, head) pairs, for `total` steps of all pairs: three
// workgroups a compute unit.  No part of under kLeastKeys keys is made, and
// no more than kPartsOfOne of the longest pair (`longest` steps), whose parts
// one workgroup joins.
constexpr int kPartsMore = 768, kLeastKeys = 1024, kPartsOfOne = 64;
KV4_HD int kv4_part_limit(int64_t total, int longest, int keys)
{
    const int64_t l = (total + kPartsMore - 1) / kPartsMore;
    const int least = kLeastKeys / keys, most = (longest + kPartsOfOne - 1) / kPartsOfOne;
    const int limit = l > 0x3fffffff ? 0x3fffffff : (int)l;
    return limit > least ? (limit > most ? limit : most) : (least > most ? least : most);
}
KV4_HD int kv4_split(int count, int parts, int i) { return (int)((int64_t)count * i / parts); }
// Workgroups for all parts of any lengths up to `most` keys a sequence.
KV4_HD int64_t kv4_decode_grid(int64_t B, int heads, int64_t most)
{
    const int64_t pairs = B * heads, each = most / kLeastKeys + 1;
    return pairs * (each - 1) < kPartsMore ? pairs * each : pairs + kPartsMore;
}

// The same for tiles of kTileRows rows: an item is a (sequence, head) pair's
// tile, a sequence's items are cut alike.  A part is at most an even share of
// a compute unit (joining large parts costs more than an uneven end), and not
// under kLeastTileKeys keys.  Parts of items that are cut number at most
// 2 kTileShares (ceil(x) < 2 x for x > 1).
constexpr int kTileRows = 128, kTileShares = 256, kLeastTileKeys = 512;
KV4_HD int kv4_tile_limit(int64_t total, int keys)
{
    const int64_t l = (total + kTileShares - 1) / kTileShares, least = kLeastTileKeys / keys;
    return l < least ? (int)least : l > 0x3fffffff ? 0x3fffffff : (int)l;
}
// Workgroups for all parts, and slots for the parts of items that are cut, of
// T rows in B sequences, `group` query heads a kv head, up to `most` keys.
struct Kv4Tiles {
    int64_t grid, slots;
};
KV4_HD Kv4Tiles kv4_prefill_tiles(int64_t T, int64_t B, int group, int heads, int64_t most)
{
    const int64_t items = (T * group / kTileRows + (B < T ? B : T)) * heads;
    const int64_t each = (most + 63) / 64 / (kLeastTileKeys / 64) + 1;   // parts of one item, at most
    Kv4Tiles t;
    t.slots = each < 2 ? 0 : items * each < 2 * kTileShares ? items * each : 2 * kTileShares;
    t.grid = items + t.slots;
    return t;
}

// Part `part` of `cuts` even ones of a sequence's steps (r.first, r.count) for a
// tile with the queries i0 .. i1: it has the steps [s0, s1), and of the tile's
// parts [part0, part0 + parts) hold any step that a query of it sees (one does
// where none is seen).
struct Kv4TilePart {
    int part0, parts, s0, s1;
};
KV4_HD Kv4TilePart kv4_tile_part(const Kv4Seq &s, bool causal, int window, int keys, int i0, int i1, const Kv4Steps &r,
                                 int cuts, int part)
{
    const int lo = kv4_lo(s, i0, window), hi = kv4_hi(s, i1, causal);
    const int width = (r.count + cuts - 1) / cuts;
    const int begin = lo / keys - r.first, past = (hi + keys - 1) / keys - r.first, end = past > begin ? past : begin;
    Kv4TilePart t;
    t.part0 = begin / width < cuts - 1 ? begin / width : cuts - 1;
    const int last = end > 0 ? (end - 1) / width : 0;
    t.parts = (last > t.part0 ? last : t.part0) - t.part0 + 1;
    t.s0 = r.first + (begin > part * width ? begin : part * width);
    t.s1 = r.first + (end < (part + 1) * width ? end : (part + 1) * width);
    return t;
}

// Whether the table's entry names a page at all.
KV4_HD bool kv4_page_ok(int page, int64_t pages) { return page >= 0 && page < pages; }

}  // namespace w4a8

// The attention kernels' integer rules for the CPU test suite.
#include "../../w4a8_int8_gemm_amd/csrc/kv4_index.h"

using namespace w4a8;

extern "C" {
void cut(int start, int end, int len, int T, int max_q, int most, int *out)
{
    const Kv4Seq s = kv4_cut(start, end, len, T, max_q, most);
    out[0] = s.q0, out[1] = s.m, out[2] = s.n;
}
int lo(int n, int m, int i, int window) { return kv4_lo(n, m, i, window); }
int hi(int n, int m, int i, int causal) { return kv4_hi(n, m, i, causal != 0); }
void steps(int m, int n, int causal, int window, int keys, int *out)
{
    const Kv4Steps r = kv4_steps(Kv4Seq{0, m, n}, causal != 0, window, keys);
    out[0] = r.first, out[1] = r.count;
}
int part_limit(int64_t total, int longest, int keys) { return kv4_part_limit(total, longest, keys); }
int split(int count, int parts, int i) { return kv4_split(count, parts, i); }
int64_t decode_grid(int64_t B, int heads, int64_t most) { return kv4_decode_grid(B, heads, most); }
int parts_more() { return kPartsMore; }
int tile_limit(int64_t total, int keys) { return kv4_tile_limit(total, keys); }
void tiles(int64_t T, int64_t B, int group, int heads, int64_t most, int64_t *out)
{
    const Kv4Tiles t = kv4_prefill_tiles(T, B, group, heads, most);
    out[0] = t.grid, out[1] = t.slots, out[2] = kTileRows;
}
int page_ok(int page, int64_t pages) { return kv4_page_ok(page, pages); }
}

// More of the attention kernels' integer rules for the CPU test suite.
#include "../../w4a8_int8_gemm_amd/csrc/kv4_index.h"

using namespace w4a8;

extern "C" {
void tile_part(int m, int n, int causal, int window, int keys, int i0, int i1, int cuts, int part, int *out)
{
    const Kv4Seq s = {0, m, n};
    const Kv4TilePart t = kv4_tile_part(s, causal != 0, window, keys, i0, i1, kv4_steps(s, causal != 0, window, keys), cuts, part);
    out[0] = t.part0, out[1] = t.parts, out[2] = t.s0, out[3] = t.s1;
}
int lo(int n, int m, int i, int window) { return kv4_lo(n, m, i, window); }
int hi(int n, int m, int i, int causal) { return kv4_hi(n, m, i, causal != 0); }
void steps(int m, int n, int causal, int window, int keys, int *out)
{
    const Kv4Steps r = kv4_steps(Kv4Seq{0, m, n}, causal != 0, window, keys);
    out[0] = r.first, out[1] = r.count;
}
}

extern "C" {
void cut_and_see(int start, int end, int len, int T, int max_q, int most, int i, int causal, int window, int *out)
{
    const Kv4Seq s = kv4_cut(start, end, len, T, max_q, most);
    const Kv4Steps r = kv4_steps(s, causal != 0, window, 32);
    out[0] = s.q0, out[1] = s.m, out[2] = kv4_lo(s, i, window), out[3] = kv4_hi(s, i, causal != 0);
    out[4] = r.first, out[5] = r.count;
}
}

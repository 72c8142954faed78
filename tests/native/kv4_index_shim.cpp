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
void steps(int m, int n, int causal, int window, int *out)
{
    const Kv4Steps r = kv4_steps(Kv4Seq{0, m, n}, causal != 0, window);
    out[0] = r.first, out[1] = r.count;
}
int64_t part_begin(int64_t U, int parts, int64_t i) { return kv4_part_begin(U, parts, i); }
int part_of(int64_t U, int parts, int64_t u) { return kv4_part_of(U, parts, u); }
int parts(int64_t U, int most, int least) { return kv4_parts(U, most, least); }
int page_ok(int page, int64_t pages) { return kv4_page_ok(page, pages); }
}

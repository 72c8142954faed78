"""Attention over the 4-bit cache in every form its kernels take: batches past a wave's 64 lanes, keys cut
into parts for every head size, windows over cut keys, and parts in a captured graph."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import w4a8_int8_gemm_amd as w  # noqa: E402
from tests.kv4_util import HEADS_AND_GROUPS, visible  # noqa: E402
from tests.test_gpu_kv4_attention import Case, dev  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [63, 64, 65, 70, 128, 130, 193])
def test_batches_past_64_sequences(n):
    """Few rows: sequences of 0 to 40 tokens, and long ones of several parts at the ends and borders."""
    kv = [(7 * b) % 41 for b in range(n)]
    for b in (0, 31, 62, 63, 64, 65, 127, 128, n - 1):
        if b < n:
            kv[b] = 1100 + b
    Case(kv, [1] * n, 4, 2, 64, 32, 16, seed=n).check(plain_decode=True)


@pytest.mark.parametrize("n", [65, 129, 150])
def test_batches_past_64_sequences_of_every_kind(n):
    """Rows for the one kernel, for the other, none at all; some cut into parts."""
    r = np.random.default_rng(n)
    m = [int(r.choice([0, 1, 3, 20])) for _ in range(n)]
    kv = [int(r.integers(0, 60)) for _ in range(n)]
    for b, (q, k) in {2: (40, 1200), 40: (1, 2100), 63: (2, 1500), 64: (33, 1300), n - 1: (17, 1100)}.items():
        m[b], kv[b] = q, k
    Case(kv, m, 4, 2, 64, 64, 16, seed=n).check()


@pytest.mark.parametrize("D,G", HEADS_AND_GROUPS)
@pytest.mark.parametrize("hq,m", [(2, [1, 1]), (8, [3, 1]), (16, [4, 3]), (4, [65, 40])])
def test_keys_cut_into_parts(D, G, hq, m):
    """1 to 16 rows, 17 to 32, and many; a few keys apart from the cuts."""
    Case([2500, 1300], m, hq, 2 if hq > 2 else 1, D, G, 64, seed=D + G + hq).check()


@pytest.mark.parametrize("hq,hk,m", [(4, 2, [600, 90]), (2, 2, [5, 3]), (8, 1, [3, 4])])
@pytest.mark.parametrize("window", [300, 700, 1500])
def test_windows_over_keys_cut_into_parts(hq, hk, m, window):
    """Tiles whose rows see none of the first parts, some parts' last and first keys, or all."""
    Case([3000, 2200], m, hq, hk, 64, 64, 32, seed=window).check(window=window)


def test_not_causal_over_keys_cut_into_parts():
    Case([2500, 90, 1300], [70, 2, 40], 4, 2, 128, 64, 16, seed=41).check(causal=False)
    Case([2500, 90, 1300], [4, 2, 1], 4, 2, 128, 64, 16, seed=41).check(causal=False)


def test_the_definition_agrees_with_the_visible_keys():
    for n, m, window in [(5, 3, 0), (5, 3, 2), (2, 4, 0), (0, 2, 3), (9, 9, 4)]:
        for i in range(m):
            lo, hi = visible(n, m, i, True, window)
            p = n - m + i
            assert [j for j in range(n) if lo <= j < hi] == [j for j in range(n) if j <= p and (not window or j > p - window)]


@pytest.mark.parametrize("m", [[1, 1], [4, 2], [70, 3]])
def test_parts_in_a_captured_graph(m):
    """The counters of the parts serve every replay; eager work and other lengths lie between them."""
    c = Case([2900, 2300], m, 8, 2, 128, 64, 16, seed=42)
    T = sum(m)
    q, table, lens, starts = dev(c.q), dev(c.table), dev(np.array(c.kv, np.int32)), dev(c.starts)
    ws = w.kv4_attention_workspace(c.c, 8, T, 2, max(m))
    other = w.kv4_attention_workspace(c.c, 8, T, 2, max(m))
    out = torch.empty((T, 8, 128), dtype=torch.float16, device="cuda")
    lse = torch.empty((T, 8), device="cuda")

    def call(workspace, out, lse):
        w.kv4_attention(q, c.c, table, lens, q_starts=starts, max_q=max(m), workspace=workspace, out=out, lse=lse)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(ws, out, lse)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(ws, out, lse)
    want, logs = torch.empty_like(out), torch.empty_like(lse)
    for k in range(5):
        lens.copy_(dev(np.array([2900 - 500 * k, 2300 - k], np.int32)))
        out.fill_(float("nan"))
        graph.replay()
        if k == 2:
            graph.replay()                                 # twice in a row, nothing between
        torch.cuda.synchronize()
        call(other, want, logs)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, logs)
        if k == 3:
            call(ws, want, logs)                           # an eager call on the graph's workspace
            ws[:4096].fill_(0x55)                          # or anything else there


@pytest.mark.parametrize("m", [[1, 1], [70, 3]])
def test_calls_in_turn_on_one_workspace(m):
    """Calls of other sizes leave their counters and parts behind."""
    a = Case([2500, 1800], m, 8, 2, 128, 64, 16, seed=43)
    b = Case([1500, 2600], m[::-1], 8, 2, 128, 64, 16, seed=44)
    ws = w.kv4_attention_workspace(a.c, 8, sum(m), 2, max(m))

    def call(c):
        return w.kv4_attention(dev(c.q), c.c, dev(c.table), dev(np.array(c.kv, np.int32)), q_starts=dev(c.starts),
                               max_q=max(m), workspace=ws, return_lse=True)

    first = [call(a), call(b)]
    for _ in range(3):
        for c, (out, lse) in zip((a, b), first):
            again, logs = call(c)
            assert torch.equal(again, out) and torch.equal(logs, lse)

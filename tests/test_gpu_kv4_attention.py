"""Attention over the 4-bit cache on the GPU against its definition in 64 bits."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import w4a8_int8_gemm_amd as w  # noqa: E402
from tests.kv4_util import HEADS_AND_GROUPS, attention, int4_rule, row_bytes, values  # noqa: E402

pytestmark = pytest.mark.gpu


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Case:
    """Sequences over a cache whose every unused byte is hostile: scales NaN, infinite or huge,
    codes arbitrary, the table's unused entries far outside."""

    def __init__(self, kv, m, hq, hk, D, G, page, seed=0, gain=1.0, bad=()):
        r = np.random.default_rng(seed)
        self.kv, self.m, self.hq, self.hk, self.D, self.G, self.page = kv, m, hq, hk, D, G, page
        per = [-(-n // page) for n in kv]
        pages = sum(per) + 2
        order = r.permutation(pages)
        self.table = np.where(r.random((len(kv), max(1, max(per)) + 1)) < 0.5, -7, 2 ** 31 - 1).astype(np.int32)
        self.c = w.KV4Cache.empty(pages, hk, page, D, G)
        hold = {n: r.integers(0, 256, (pages, hk, page, D // 2)).astype(np.uint8) for n in "kv"}
        scales = {n: r.choice(np.array([np.nan, np.inf, -np.inf, 3e38], np.float32), (pages, hk, page, D // G))
                  for n in "kv"}
        self.k, self.v, self.there = [], [], []
        at = 0
        for b, n in enumerate(kv):
            self.table[b, :per[b]] = order[at:at + per[b]]
            at += per[b]
            real = {}
            for name in "kv":
                x = (gain * r.standard_normal((n, hk, D))).astype(np.float16)
                if name == "k":
                    x[..., 3::29] *= 4
                q, s = int4_rule(x, G)
                real[name] = values(q, s, G)
                j = np.arange(n)
                p = self.table[b, j // page]
                hold[name][p, :, j % page] = row_bytes(q, name)
                scales[name][p, :, j % page] = s
            self.k.append(real["k"])
            self.v.append(real["v"])
            self.there.append(np.ones(n, bool))
        for b, p, entry in bad:                            # pages that are not there
            self.table[b, p] = entry if entry < 0 else pages + entry
            self.there[b][p * page:(p + 1) * page] = False
        self.c.k.copy_(dev(hold["k"]))
        self.c.v.copy_(dev(hold["v"]))
        self.c.k_scale.copy_(dev(scales["k"]))
        self.c.v_scale.copy_(dev(scales["v"]))
        self.starts = np.concatenate(([0], np.cumsum(m))).astype(np.int32)
        self.q = r.standard_normal((sum(m), hq, D)).astype(np.float16)

    def run(self, causal=True, window=0, scale=None, plain_decode=False, q=None, **kw):
        T = sum(self.m)
        ws = w.kv4_attention_workspace(self.c, self.hq, T, len(self.kv), max(self.m))
        ws.fill_(0xFF)                                     # nothing in it is relied on
        out = torch.full((T, self.hq, self.D), float("nan"), dtype=torch.float16, device="cuda")
        lse = torch.full((T, self.hq), float("nan"), device="cuda")
        args = {} if plain_decode else dict(q_starts=dev(self.starts), max_q=max(self.m))
        w.kv4_attention(dev(self.q) if q is None else q, self.c, dev(self.table),
                        dev(np.array(self.kv, np.int32)), causal=causal, window=window, scale=scale,
                        workspace=ws, out=out, lse=lse, **args, **kw)
        return out, lse

    def check(self, causal=True, window=0, scale=None, **kw):
        out, lse = self.run(causal, window, scale, **kw)
        out, lse = out.cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
        for b in range(len(self.kv)):
            rows = slice(self.starts[b], self.starts[b + 1])
            want, logs, ob, lb = attention(self.q[rows], self.k[b], self.v[b], self.there[b], None, None,
                                           causal, window, self.D ** -0.5 if scale is None else scale, self.page)
            assert np.isfinite(out[rows]).all(), f"sequence {b}: not finite"
            assert (np.abs(out[rows] - want) <= ob).all(), \
                f"sequence {b}: {float((np.abs(out[rows] - want) / ob).max()):.3g} of the bound"
            none = np.isinf(logs)
            assert (lse[rows][none] == -np.inf).all() and (out[rows][none] == 0).all()
            assert (np.abs(lse[rows] - logs)[~none] <= lb[~none]).all()
        return out


@pytest.mark.parametrize("D,G", HEADS_AND_GROUPS)
def test_one_token_a_sequence(D, G):
    kv = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 300, 517]
    Case(kv, [1] * len(kv), 8, 2, D, G, 16, seed=D + G).check(plain_decode=True)


@pytest.mark.parametrize("hq,hk", [(1, 1), (3, 1), (4, 4), (7, 1), (14, 2), (16, 1), (17, 1), (32, 8), (40, 1),
                                   (71, 1), (15, 5)])
def test_head_layouts(hq, hk):
    kv = [200, 33, 1]
    Case(kv, [1] * 3, hq, hk, 128, 64, 32, seed=hq).check()


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256, 1024])
@pytest.mark.parametrize("D,G", [(64, 64), (128, 32), (256, 128)])
def test_pages(page, D, G):
    kv = [page - 1, page, page + 1, 2 * page + 13]
    Case(kv, [1, 2, 1, 3], 4, 2, D, G, page, seed=page).check()


@pytest.mark.parametrize("m", [[2, 1, 5], [4, 4, 4], [16, 3, 9], [1, 0, 17], [33, 40, 1], [0, 0, 1]])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D,G", [(64, 32), (128, 128), (256, 64)])
def test_several_queries(m, causal, D, G):
    Case([50, 130, 77], m, 8, 2, D, G, 16, seed=sum(m)).check(causal)


@pytest.mark.parametrize("D,G", HEADS_AND_GROUPS)
@pytest.mark.parametrize("causal", [True, False])
def test_many_queries(D, G, causal):
    Case([150, 97, 260, 64], [150, 70, 33, 64], 4, 2, D, G, 16, seed=D * G).check(causal)


@pytest.mark.parametrize("hq,hk,m,kv", [(1, 1, [129], [129]), (6, 2, [43, 1], [300, 90]), (5, 1, [100], [100]),
                                        (7, 1, [64, 65], [70, 65]), (16, 2, [32, 8], [45, 200]),
                                        (24, 3, [90], [400])])
def test_many_queries_head_layouts(hq, hk, m, kv):
    Case(kv, m, hq, hk, 128, 64, 16, seed=hq).check()


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 33, 64, 100, 1000])
@pytest.mark.parametrize("m", [[1, 1, 1], [3, 9, 1], [60, 33, 80]])
def test_window(window, m):
    Case([120, 257, 80], m, 4, 2, 128, 64, 16, seed=window).check(window=window)


@pytest.mark.parametrize("m", [[5, 9, 2], [40, 70, 33]])
@pytest.mark.parametrize("window", [0, 3])
def test_rows_that_see_nothing(m, window):
    """More queries than keys: the first ones stand before the first key."""
    Case([0, 4, 1], m, 4, 2, 128, 128, 16, seed=3).check(window=window)


@pytest.mark.parametrize("m", [[1, 1], [3, 2], [50, 120]])
def test_pages_that_are_not_there(m):
    """Tokens of pages outside the cache are not seen; a sequence without any page sees nothing."""
    c = Case([140, 130], m, 4, 2, 128, 64, 16, seed=4,
             bad=[(0, 0, -1), (0, 3, 0), (0, 7, 2 ** 30), (1, 8, -2 ** 31)])
    c.check()
    c.check(causal=False)
    c = Case([33, 20], m, 4, 2, 64, 32, 16, seed=4, bad=[(0, 0, -1), (0, 1, -2), (0, 2, 5)])
    c.check(causal=False)


def test_tables_past_their_buffers():
    """Lengths past the table's pages and query ranges past the rows are cut."""
    c = Case([40, 40], [1, 1], 4, 2, 64, 64, 16, seed=5)
    good, _ = c.run()
    table = c.table[:, :3]
    lens = np.array([2 ** 31 - 1, -5], np.int32)
    out = w.kv4_attention(dev(c.q), c.c, dev(table), dev(lens), causal=False)
    # 48 slots of the first sequence: its 40 tokens and 8 hostile ones, so only finite inputs say something
    assert bool((out[1] == 0).all())
    starts = np.array([0, 1, 2 ** 31 - 1], np.int32)
    again = w.kv4_attention(dev(c.q), c.c, dev(c.table), dev(np.array(c.kv, np.int32)), q_starts=dev(starts), max_q=1)
    assert torch.equal(again, good)
    starts = np.array([-9, 1, 2], np.int32)
    w.kv4_attention(dev(c.q), c.c, dev(c.table), dev(np.array(c.kv, np.int32)), q_starts=dev(starts), max_q=2)
    torch.cuda.synchronize()


@pytest.mark.parametrize("gain,scale", [(0.01, None), (30.0, None), (1.0, 3.0), (1e-4, 1.0), (300.0, 1e-3)])
@pytest.mark.parametrize("m", [[1, 2], [90, 40]])
def test_sizes_of_values(gain, scale, m):
    """Flat and peaked softmax, values near fp16's ends."""
    Case([300, 129], m, 4, 2, 128, 32, 16, seed=6, gain=gain).check(scale=scale)


def test_values_of_very_different_tokens():
    """Tokens whose values differ by 2^20, the heavy ones' weights small."""
    c = Case([256], [3], 4, 2, 128, 128, 16, seed=7)
    s = c.c.v_scale.cpu().numpy()
    f = np.float32(2.0) ** np.random.default_rng(0).integers(-20, 1, 256)
    for j in range(256):
        s[c.table[0, j // 16], :, j % 16] *= f[j]
        c.v[0][j] *= f[j]
    c.c.v_scale.copy_(dev(s))
    c.check()


def test_all_values_zero_and_queries_zero():
    c = Case([100, 70], [1, 40], 4, 2, 64, 64, 16, seed=8)
    c.q[:] = 0
    c.check()
    c.c.v.zero_()
    c.c.v_scale.zero_()
    for v in c.v:
        v[:] = 0
    out = c.check()
    assert (out == 0).all()


@pytest.mark.parametrize("kv,m,hq,hk", [([5000], [1], 8, 2), ([3001, 40, 2222, 700], [1, 1, 1, 1], 4, 4),
                                        ([4097], [5], 8, 1), ([2500], [130], 2, 1)])
def test_long_sequences_are_split(kv, m, hq, hk):
    Case(kv, m, hq, hk, 128, 128, 64, seed=9).check()


def test_the_same_call_gives_the_same_bits():
    c = Case([3000, 77, 1500], [1, 1, 1], 8, 2, 128, 64, 16, seed=10)
    a, la = c.run()
    for _ in range(3):
        b, lb = c.run()
        assert torch.equal(a, b) and torch.equal(la, lb)


def test_one_query_a_sequence_with_and_without_starts():
    c = Case([300, 20], [1, 1], 8, 2, 128, 64, 16, seed=11)
    a, la = c.run()
    b, lb = c.run(plain_decode=True)
    assert torch.equal(a, b) and torch.equal(la, lb)


@pytest.mark.parametrize("m", [[1, 1], [70, 33]])
def test_strided_queries_and_another_stream(m):
    c = Case([150, 90], m, 8, 2, 128, 64, 16, seed=12)
    a, la = c.run()
    T = sum(m)
    qkv = torch.full((T, 12, 128), float("nan"), dtype=torch.float16, device="cuda")
    qkv[:, :8] = dev(c.q)
    b, lb = c.run(q=qkv[:, :8])
    assert torch.equal(a, b) and torch.equal(la, lb)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        b, lb = c.run()
    st.synchronize()
    assert torch.equal(a, b) and torch.equal(la, lb)


def test_non_finite_queries_stay_in_their_row():
    c = Case([60, 60], [1, 40], 4, 2, 64, 64, 16, seed=13)
    good, _ = c.run()
    c.q[0, 1] = np.nan
    c.q[7, 2, 5] = np.inf
    out, _ = c.run()
    keep = torch.ones(41, 4, dtype=torch.bool)
    keep[0, 1] = keep[7, 2] = False
    assert torch.equal(out[keep.cuda()], good[keep.cuda()])


@pytest.mark.parametrize("m", [[1, 1, 1], [40, 2, 9]])
def test_graph_replays(m):
    """A captured call follows the lengths that the buffers hold at each replay."""
    c = Case([900, 333, 64], m, 8, 2, 128, 64, 16, seed=14)
    T = sum(m)
    q, table, lens, starts = dev(c.q), dev(c.table), dev(np.array(c.kv, np.int32)), dev(c.starts)
    ws = w.kv4_attention_workspace(c.c, 8, T, 3, max(m))
    out = torch.empty((T, 8, 128), dtype=torch.float16, device="cuda")
    lse = torch.empty((T, 8), device="cuda")

    def call():
        w.kv4_attention(q, c.c, table, lens, q_starts=starts, max_q=max(m), workspace=ws, out=out, lse=lse)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for k in range(4):
        new = np.array([900 - 61 * k, 333 - 7 * k, 64 - k], np.int32)
        lens.copy_(dev(new))
        graph.replay()
        torch.cuda.synchronize()
        got, logs = out.clone(), lse.clone()
        ws.fill_(0x7F)
        call()
        torch.cuda.synchronize()
        assert torch.equal(got, out) and torch.equal(logs, lse)


def test_no_rows():
    c = Case([5], [1], 4, 2, 64, 64, 16)
    q = torch.empty((0, 4, 64), dtype=torch.float16, device="cuda")
    z = torch.zeros((1,), dtype=torch.int32, device="cuda")
    out, lse = w.kv4_attention(q, c.c, torch.empty((0, 0), dtype=torch.int32, device="cuda"), z[:0], return_lse=True)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    # a sequence without pages: its query sees nothing
    q = torch.randn(1, 4, 64, device="cuda").half()
    out, lse = w.kv4_attention(q, c.c, torch.empty((1, 0), dtype=torch.int32, device="cuda"), z + 9, return_lse=True)
    assert bool((out == 0).all()) and bool((lse == float("-inf")).all())


def test_a_cache_past_32_bits():
    """Pages whose rows lie over 4 GiB into the buffers, one page of 2^16 tokens a sequence."""
    D, G, page, hk = 128, 64, 1 << 16, 8
    pages = (4 << 30) // (page * hk * D // 2) + 2
    c = w.KV4Cache.empty(pages, hk, page, D, G)
    assert c.k.numel() > 1 << 32
    small = w.KV4Cache.empty(64, hk, 16, D, G)
    k = torch.randn(1000, hk, D, device="cuda").half()
    v = torch.randn(1000, hk, D, device="cuda").half()
    at = torch.arange(1000, device="cuda")
    w.kv4_write(k, v, at + (pages - 1) * page, c)
    w.kv4_write(k, v, at, small)
    lens = torch.tensor([1000], dtype=torch.int32, device="cuda")
    for m in (1, 50):
        q = torch.randn(m, 16, D, device="cuda").half()
        starts = torch.tensor([0, m], dtype=torch.int32, device="cuda")
        a = w.kv4_attention(q, c, torch.tensor([[pages - 1]], dtype=torch.int32, device="cuda"), lens, starts, m)
        # the other table's pages allow fewer splits; the results agree to the fp16 rounding of two sums
        b = w.kv4_attention(q, small, torch.arange(63, dtype=torch.int32, device="cuda")[None], lens, starts, m)
        assert float((a.float() - b.float()).abs().max()) <= 2.0 ** -9 * float(v.abs().max())

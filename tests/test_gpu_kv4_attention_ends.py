"""Attention over the 4-bit cache where its arguments and its cache are at their ends, against the
definition in 64 bits."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import w4a8_int8_gemm_amd as w  # noqa: E402
from tests.kv4_util import attention  # noqa: E402
from tests.test_gpu_kv4_attention import Case, dev  # noqa: E402

pytestmark = pytest.mark.gpu

TOP = 2 ** 31 - 1


@pytest.mark.parametrize("kv,m", [([0, 4, 1], [5, 9, 2]), ([0, 4, 1], [40, 70, 33]), ([3, 100, 1], [200, 150, 300])])
@pytest.mark.parametrize("window", [TOP, TOP - 1, 2 ** 30])
def test_the_largest_windows(kv, m, window):
    """More queries than keys, so that the first key of a window lies below -2^31."""
    Case(kv, m, 4, 2, 128, 128, 16, seed=21).check(window=window)


HOSTILE = {"nan": np.nan, "inf": np.inf, "-inf": -np.inf, "huge": 3e38, "-huge": -3e38, "mixed": None}


def spoil(c, b, keys, kind, names="kv", groups=slice(None), seed=0):
    """Hostile scales and arbitrary codes for some keys of sequence b."""
    r = np.random.default_rng(seed)
    for name in names:
        codes, scales = getattr(c.c, name), getattr(c.c, name + "_scale")
        for j in keys:
            page, at = int(c.table[b, j // c.page]), j % c.page
            codes[page, :, at] = dev(r.integers(0, 256, (c.hk, c.D // 2)).astype(np.uint8))
            value = HOSTILE[kind] if kind != "mixed" else r.choice([np.nan, np.inf, -np.inf, 3e38, -3e38, -1.0])
            scales[page, :, at, groups] = float(value)


def check_rows(c, rows_of, causal=True, window=0):
    """The rows that rows_of gives for a sequence, against the definition."""
    out, lse = c.run(causal, window)
    out, lse = out.cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    for b in range(len(c.kv)):
        first = c.starts[b]
        want, logs, ob, lb = attention(c.q[first:c.starts[b + 1]], c.k[b], c.v[b], c.there[b], None, None, causal, window,
                                       c.D ** -0.5, c.page)
        for i in rows_of(b):
            got = out[first + i]
            assert np.isfinite(got).all(), f"sequence {b} row {i}: not finite"
            assert (np.abs(got - want[i]) <= ob[i]).all(), f"sequence {b} row {i}"
            same = logs[i] == lse[first + i]
            with np.errstate(invalid="ignore"):
                assert (same | (np.abs(lse[first + i] - logs[i]) <= lb[i])).all(), f"sequence {b} row {i}"
    return out, lse


@pytest.mark.parametrize("kind", HOSTILE)
@pytest.mark.parametrize("page", [16, 32])
@pytest.mark.parametrize("m", [[1, 1, 1], [3, 8, 1], [60, 33, 80]])
def test_keys_behind_the_window_have_no_influence(m, page, kind):
    """What lies in front of every query's window may be anything: its page may have been given away."""
    for D, G, window in ((128, 64, 50), (64, 64, 17), (256, 64, 33), (128, 128, 1)):
        c = Case([120, 257, 80], m, 4, 2, D, G, page, seed=22)
        for b, (n, q) in enumerate(zip(c.kv, m)):
            spoil(c, b, range(max(0, n - q + 1 - window)), kind)
        check_rows(c, lambda b: range(m[b]), window=window)


@pytest.mark.parametrize("kind", HOSTILE)
@pytest.mark.parametrize("names", ["k", "v"])
@pytest.mark.parametrize("m", [[5, 2], [8, 16], [70, 140]])
def test_a_later_token_does_not_change_an_earlier_row(m, names, kind):
    """The last token's key and value are seen by the last query alone."""
    for D, G in ((128, 64), (64, 64), (256, 128)):
        c = Case([75, 140], m, 4, 2, D, G, 16, seed=23)
        for b, n in enumerate(c.kv):
            spoil(c, b, [n - 1], kind, names)
        check_rows(c, lambda b: range(m[b] - 1))


@pytest.mark.parametrize("kind", HOSTILE)
@pytest.mark.parametrize("m", [[6, 3], [50, 70]])
def test_a_token_that_left_the_window_does_not_change_a_row(m, kind):
    """The first query alone still sees the key that is spoiled."""
    c = Case([90, 200], m, 8, 2, 128, 32, 16, seed=24)
    for b, (n, q) in enumerate(zip(c.kv, m)):
        spoil(c, b, [max(0, n - q + 1 - 20)], kind)
    check_rows(c, lambda b: range(1 if c.kv[b] - m[b] + 1 >= 20 else m[b], m[b]), window=20)


@pytest.mark.parametrize("m", [[1], [4], [60]])
@pytest.mark.parametrize("causal", [True, False])
def test_a_seen_value_that_is_not_finite_stays_in_its_group(m, causal):
    """Rows that see it are not finite in the elements of its scale group, and as they are in the others."""
    c = Case([77], m, 4, 2, 128, 32, 16, seed=25)
    good, logs = (t.cpu().numpy() for t in c.run(causal))
    j = 76 - m[0] // 2
    page, at = int(c.table[0, j // 16]), j % 16
    c.c.v_scale[page, 1, at, 2] = float("nan")
    out, lse = (t.cpu().numpy() for t in c.run(causal))
    sees = np.arange(m[0]) + 77 - m[0] >= j if causal else np.ones(m[0], bool)
    touched = np.zeros(out.shape, bool)
    touched[np.ix_(sees, [2, 3], np.arange(64, 96))] = True
    assert np.isnan(out[touched]).all() and sees.any()
    # the other elements: the reference of the weights may differ, two roundings to fp16 on each side
    assert (np.abs(out.astype(float) - good)[~touched] <= 4 * 2.0 ** -11 * 8).all()
    assert np.array_equal(lse, logs) or (np.abs(lse - logs) <= 64 * 2.0 ** -24 * (1 + np.abs(logs))).all()


@pytest.mark.parametrize("m", [[1, 5, 8], [70, 33, 64]])
def test_values_far_larger_than_what_an_earlier_row_sees(m):
    """A later token's values are 2^16 times the others, all within fp16."""
    c = Case([90, 130, 64], m, 4, 2, 128, 64, 16, seed=26, gain=0.01)
    for b, n in enumerate(c.kv):
        page, at = int(c.table[b, (n - 1) // 16]), (n - 1) % 16
        c.c.v_scale[page, :, at] *= 2.0 ** 16
        c.v[b][n - 1] *= 2.0 ** 16
    check_rows(c, lambda b: range(m[b]))


@pytest.mark.parametrize("m,most", [([6, 3], 4), ([6, 3], 1), ([70, 5], 40), ([70, 200], 64), ([33, 2], 3)])
@pytest.mark.parametrize("window", [0, 9])
def test_rows_past_max_q_are_not_computed_and_do_not_move_the_others(m, most, window):
    c = Case([100, 210], m, 8, 2, 128, 64, 16, seed=27)
    T = sum(m)
    out = torch.full((T, 8, 128), float("nan"), dtype=torch.float16, device="cuda")
    lse = torch.full((T, 8), float("nan"), device="cuda")
    w.kv4_attention(dev(c.q), c.c, dev(c.table), dev(np.array(c.kv, np.int32)), q_starts=dev(c.starts), max_q=most,
                    window=window, out=out, lse=lse)
    out, lse = out.cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    for b in range(2):
        rows = slice(c.starts[b], c.starts[b + 1])
        want, logs, ob, lb = attention(c.q[rows], c.k[b], c.v[b], c.there[b], None, None, True, window, 128 ** -0.5, 16)
        kept = min(m[b], most)
        assert (np.abs(out[rows] - want) <= ob)[:kept].all() and (np.abs(lse[rows] - logs) <= lb)[:kept].all()
        assert np.isnan(out[rows][kept:]).all() and np.isnan(lse[rows][kept:]).all()


@pytest.mark.parametrize("n", [70001, 131075])
@pytest.mark.parametrize("m,hq", [(1, 8), (2, 8), (40, 2)])
def test_zero_values_of_many_keys(n, m, hq):
    """All scores are 0: the log of the sum is log n; then values behind n - 4000 zero ones."""
    page, D, G = 1024, 64, 32
    pages = -(-n // page)
    c = w.KV4Cache.empty(pages, 1, page, D, G)
    for t in (c.k, c.v, c.k_scale, c.v_scale):
        t.zero_()
    q = torch.zeros((m, hq, D), dtype=torch.float16, device="cuda")
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, m], dtype=torch.int32, device="cuda")

    def call():
        out, lse = w.kv4_attention(q, c, table, lens, q_starts=starts, max_q=m, causal=False, return_lse=True)
        # a sum of n ones in fp32: n u; the log and its factor a few steps
        assert bool(((lse.double() - float(np.log(n))).abs() <= n * 2.0 ** -24 + 64 * 2.0 ** -24).all())
        return out.double()

    assert bool((call() == 0).all())
    at = torch.arange(n - 4000, n, device="cuda")
    c.v[at // page, 0, at % page] = 0x77
    c.v_scale[at // page, 0, at % page] = 2.0
    want = 14.0 * 4000 / n
    # the output's rounding and the weights', and the two sums
    assert bool(((call() - want).abs() <= want * (2 * 2.0 ** -11 + 2 * n * 2.0 ** -24)).all())


@pytest.mark.parametrize("m", [1, 40])
@pytest.mark.parametrize("exponent", [-24, -27, -36])
def test_the_smallest_values(m, exponent):
    """Scales down to the smallest that the writer makes (2^-24 / 7), and below: what fp16 holds of them."""
    c = Case([90], [m], 4, 2, 64, 32, 16, seed=28)
    f = np.float32(2.0) ** exponent
    c.c.v_scale.mul_(float(f))
    c.v[0] = c.v[0] * float(f)
    check_rows(c, lambda b: range(m))


@pytest.mark.parametrize("hq,hk", [(8, 2), (40, 1)])
@pytest.mark.parametrize("scale", [1e28, 1e31, 1e36, 2.0 ** 120])
def test_scores_far_below_zero(hq, hk, scale):
    """A row's only key has all its weight whatever its score is (|scores| up to about 2^125)."""
    c = Case([1, 1, 1, 1], [1, 1, 1, 1], hq, hk, 64, 32, 16, seed=29)
    out = c.check(scale=scale)
    for b in range(4):
        v = np.repeat(c.v[b][0], hq // hk, 0)
        assert (np.abs(out[b] - v) <= 2 * 2.0 ** -11 * np.abs(v) + 2.0 ** -25).all()


@pytest.mark.parametrize("m", [[1, 3], [40, 70]])
@pytest.mark.parametrize("gain,scale", [(1e-3, s) for s in (1e7, 1e8, 1e9, 4e9, 1e10, 3e10, 1e11, 1e12)] +
                         [(1.0, 1e6), (1.0, 1e7), (1e-6, 1e14), (100.0, 1e4), (1000.0, 1e3)])
def test_scores_whose_steps_are_larger_than_one(m, gain, scale):
    """Scores past 2^24, which fp32 holds in steps of 2 and more: one key has all the weight."""
    c = Case([300, 129], m, 4, 2, 128, 32, 16, seed=30, gain=gain)
    out = c.check(scale=scale)
    first = 0
    for b, q in enumerate(m):
        for i in range(q):
            n = c.kv[b] - q + i + 1
            for h in range(4):
                s = c.k[b][:n, h // 2] @ c.q[first + i, h].astype(np.float64) * scale
                top = np.argsort(s)[-2:]
                reach = (np.abs(c.k[b][:n, h // 2]) @ np.abs(c.q[first + i, h].astype(np.float64))).max() * scale
                if s[top[1]] - s[top[0]] > 2 * (128 + 8) * 2.0 ** -23 * reach + 40:    # a second key's weight is under e^-40
                    v = c.v[b][top[1], h // 2]
                    assert (np.abs(out[first + i, h] - v) <= 2 * 2.0 ** -11 * np.abs(v) + 16 * 2.0 ** -25).all()
        first += q


def check_two_part_weights(c, out, causal=True, window=0):
    """The bound of the definition with weights of 22 bits: p |v| is the output of |v|."""
    for b in range(len(c.kv)):
        rows = slice(c.starts[b], c.starts[b + 1])
        args = (c.there[b], None, None, causal, window, c.D ** -0.5, c.page)
        want, _, ob, _ = attention(c.q[rows], c.k[b], c.v[b], *args)
        reach = attention(c.q[rows], c.k[b], np.abs(c.v[b]), *args)[0]
        tight = ob - (2.0 ** -11 - 2.0 ** -22) * 1.01 * reach
        assert (np.abs(out[rows] - want) <= tight).all(), float((np.abs(out[rows] - want) / tight).max())


@pytest.mark.parametrize("kv,m,window", [([900, 30], [1, 3], 0), ([5000], [1], 16), ([5000, 2000], [5, 1], 100),
                                         ([3000], [4], 1024), ([1024 + 3], [4], 0)])
def test_weights_have_22_bits_where_a_row_sees_few_keys(kv, m, window):
    """Few keys seen, not few keys in the cache: a window behind a long context counts as a short one."""
    c = Case(kv, m, 4, 2, 128, 64, 16, seed=31)
    c.q[:] = 0                                            # equal weights: no error of the scores hides their rounding
    c.check(window=window)
    out, _ = c.run(window=window)
    check_two_part_weights(c, out.cpu().numpy().astype(np.float64), window=window)


@pytest.mark.parametrize("m", [[1, 1, 1], [3, 1, 0], [40, 2, 7]])
def test_a_buffer_of_full_size_with_shorter_ranges(m):
    """As a captured call has it: rows for max_q queries of every sequence, q_starts gives fewer; the rows
    of no sequence are not written."""
    c = Case([100, 210, 64], m, 8, 2, 128, 64, 16, seed=32)
    T, most = 3 * 40, 40
    q = torch.full((T, 8, 128), float("nan"), dtype=torch.float16, device="cuda")
    q[:sum(m)] = dev(c.q)
    out = torch.full((T, 8, 128), float("nan"), dtype=torch.float16, device="cuda")
    lse = torch.full((T, 8), float("nan"), device="cuda")
    w.kv4_attention(q, c.c, dev(c.table), dev(np.array(c.kv, np.int32)), q_starts=dev(c.starts), max_q=most, out=out,
                    lse=lse)
    out, lse = out.cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    for b in range(3):
        rows = slice(c.starts[b], c.starts[b + 1])
        want, logs, ob, lb = attention(c.q[rows], c.k[b], c.v[b], c.there[b], None, None, True, 0, 128 ** -0.5, 16)
        assert (np.abs(out[rows] - want) <= ob).all() and (np.abs(lse[rows] - logs) <= lb).all()
    assert np.isnan(out[sum(m):]).all() and np.isnan(lse[sum(m):]).all()


@pytest.mark.parametrize("m", [[5, 3], [70, 40]])
def test_without_max_q_every_row_is_computed(m):
    """q_starts alone says how many queries a sequence has."""
    c = Case([100, 90], m, 8, 2, 128, 64, 16, seed=33)
    good, logs = c.run()
    args = dev(c.q), c.c, dev(c.table), dev(np.array(c.kv, np.int32))
    out, lse = w.kv4_attention(*args, q_starts=dev(c.starts), return_lse=True)
    assert torch.equal(out, good) and torch.equal(lse, logs)
    ws = w.kv4_attention_workspace(c.c, 8, sum(m), 2)     # of one query a sequence: too small is said, not taken
    if max(m) * 4 > 32:
        with pytest.raises(w.W4A8Error, match="workspace"):
            w.kv4_attention(*args, q_starts=dev(c.starts), workspace=ws)


@pytest.mark.parametrize("m", [[1, 3], [40, 60]])
@pytest.mark.parametrize("name", ["k", "v"])
@pytest.mark.parametrize("D,G", [(64, 64), (128, 32), (256, 128)])
def test_negative_scales(m, name, D, G):
    """A value is code * scale, whatever the sign: some keys' scales in some groups are turned."""
    c = Case([77, 130], m, 4, 2, D, G, 16, seed=34)
    r = np.random.default_rng(5)
    for b, n in enumerate(c.kv):
        for j in range(0, n, 3):
            page, at, g = int(c.table[b, j // 16]), j % 16, int(r.integers(0, D // G))
            getattr(c.c, name + "_scale")[page, :, at, g] *= -1
            getattr(c, name)[b][j, :, g * G:(g + 1) * G] *= -1
    c.check()


@pytest.mark.parametrize("m", [1, 40])
@pytest.mark.parametrize("bits", [0x7fc00000, 0xffffffff, 0xffc00001])
def test_a_key_scale_that_is_not_a_number_makes_the_rows_that_see_it_not_a_number(m, bits):
    c = Case([77], [m], 4, 2, 128, 64, 16, seed=35)
    good, _ = c.run()
    page, at = int(c.table[0, 70 // 16]), 70 % 16
    c.c.k_scale.view(torch.int32)[page, 1, at, 0] = bits - 2 ** 32 if bits >= 2 ** 31 else bits
    out, lse = c.run()
    sees = torch.arange(m, device="cuda") + 77 - m >= 70
    assert bool(out[sees][:, 2:].isnan().all()) and bool(sees.any())
    assert torch.equal(out[:, :2], good[:, :2]) and torch.equal(out[~sees], good[~sees])


@pytest.mark.parametrize("kv,m", [([77], [1]), ([77], [40]), ([3000], [2]), ([3000], [150])])
@pytest.mark.parametrize("bad", [np.nan, np.inf])
def test_the_log_of_a_row_that_is_not_a_number(kv, m, bad):
    """Not the log of a row that sees nothing; also where its keys are cut into parts."""
    c = Case(kv, m, 4, 2, 128, 64, 16, seed=36)
    good, logs = c.run()
    last = sum(m) - 1
    c.q[last, 1, 5] = bad
    out, lse = c.run()
    assert bool(lse[last, 1].isnan()) and bool(out[last, 1].isnan().all())
    keep = torch.ones(lse.shape, dtype=torch.bool)
    keep[last, 1] = False
    assert torch.equal(lse[keep.cuda()], logs[keep.cuda()]) and torch.equal(out[keep.cuda()], good[keep.cuda()])
    page, at = int(c.table[0, 50 // 16]), 50 % 16                # in the first of the parts
    c = Case(kv, m, 4, 2, 128, 64, 16, seed=36)
    c.c.k_scale[page, 0, at] = float("nan")
    out, lse = c.run()
    sees = torch.arange(m[0], device="cuda") + kv[0] - m[0] >= 50
    assert bool(lse[sees][:, :2].isnan().all()) and bool(out[sees][:, :2].isnan().all())
    assert torch.equal(lse[:, 2:], logs[:, 2:]) and torch.equal(lse[~sees], logs[~sees])


@pytest.mark.parametrize("kv,m,window", [([75, 300], [6, 4], 0), ([75, 300], [50, 140], 0), ([75, 1300], [20, 90], 40),
                                         ([2300, 1100], [8, 2], 0), ([2300], [200], 700)])
@pytest.mark.parametrize("gain", [1e-3, 1.0, 1e4])
def test_earlier_rows_keep_their_bits(kv, m, window, gain):
    """Whatever the last token's key and value are, the rows before it come out the same to the bit."""
    c = Case(kv, m, 8, 2, 128, 64, 16, seed=37)
    good, logs = c.run(window=window)
    for b, n in enumerate(kv):
        page, at = int(c.table[b, (n - 1) // 16]), (n - 1) % 16
        for name in "kv":
            getattr(c.c, name)[page, :, at] ^= 0x35
            getattr(c.c, name + "_scale")[page, :, at] *= gain
    out, lse = c.run(window=window)
    keep = torch.ones(sum(m), dtype=torch.bool, device="cuda")
    keep[torch.from_numpy(c.starts[1:] - 1).long().cuda()] = False
    assert torch.equal(out[keep], good[keep]) and torch.equal(lse[keep], logs[keep])
    assert not torch.equal(out[~keep], good[~keep])

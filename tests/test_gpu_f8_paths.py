"""The 8-bit floating point products at sizes that reach every kernel, at sizes beyond 2^31, with workspaces
as a program has them, and the operators together as a feed-forward block."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import w4a8_int8_gemm_amd as w  # noqa: E402
from tests.f8_paths import GATED, PRODUCTS  # noqa: E402
from tests.f8_util import F8_ROUND, F8_TINY, HALF_ROUND, HALF_TINY, U  # noqa: E402

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn


def rng(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def operands(m, n, k, seed, sides=1):
    """Codes as quantised rows have them and scales of many sizes, some zero: sums of the size of 1."""
    g = rng(seed)
    kb = -(-k // 128)

    def codes(r):
        return (torch.randn(r, k, device="cuda", generator=g) * 110).clamp(-448, 448).to(F8)

    sx = (torch.randn(kb, m, device="cuda", generator=g) * 0.5).exp()
    sx[torch.rand(kb, m, device="cuda", generator=g) < 0.05] = 0
    out = [codes(m), sx]
    for _ in range(sides):
        sw = (torch.randn(-(-n // 128), kb, device="cuda", generator=g) * 0.5).exp() / (110 * 110 * math.sqrt(k))
        out += [codes(n), sw]
    return out


def parts(q, scale, weights):
    """Of every element: its value; of every eight: the scale times the power of two they are aligned by (at
    most: that of the largest field, 2^-6 for subnormals)."""
    v = q.double()
    k = q.shape[1]
    s = scale.double().repeat_interleave(128, 1)[:, :k]
    if weights:
        s = s.repeat_interleave(128, 0)[:q.shape[0]]
    field = (q.view(torch.uint8).to(torch.int32) >> 3) & 15
    e = torch.exp2((field - 7).clamp(min=-6).double())
    return v * s, (e.view(-1, k // 8, 8).amax(2)) * s[:, ::8]


def product(xq, sx, wq, sw):
    """The sums in 64 bits and how far an fp32 accumulation may be: seven of eight aligned products lose what
    lies below 2^-13 of the largest's power; fp32 additions of the groups and blocks; the scales' product."""
    xv, xe = parts(xq, sx.t(), False)
    wv, we = parts(wq, sw, True)
    out = xv @ wv.t().contiguous()
    loss = (xe @ we.t().contiguous()) * (7 * 2.0 ** -13)
    reach = xv.abs() @ wv.abs().t().contiguous()
    return out, loss + (-(-xq.shape[1] // 128) + 40) * 2 * U * reach


def activation(g, kind):
    if kind == "silu":
        return g / (1 + torch.exp(-g))
    return 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)))


def gated(xq, sx, wg, sg, wu, su, kind):
    """In 64 bits; the slope of either activation lies below 1.13, its fp32 evaluation is good to 2^-20."""
    g, dg = product(xq, sx, wg, sg)
    u, du = product(xq, sx, wu, su)
    assert g.abs().amax() <= 60
    a = activation(g, kind)
    da = 1.13 * dg + 2.0 ** -20 * a.abs()
    return a * u, da * (u.abs() + du) + a.abs() * du + 2 * U * (a * u).abs()


def check_half(y, v, dv):
    assert ((y.double() - v).abs() <= dv + (v.abs() + dv) * HALF_ROUND * 1.001 + HALF_TINY).all()


def check_codes(q, s, v, dv):
    """Each block's scale, then every code: half a step of the code's value (or of the subnormals below 2^-6 of
    the scale), the quotient's rounding, what v itself is off by and what the scale is."""
    n = v.shape[1]
    pad = torch.nn.functional.pad
    top = pad(v.abs(), (0, -n % 128)).view(v.shape[0], -1, 128).amax(2).t()
    far = pad(dv, (0, -n % 128)).view(v.shape[0], -1, 128).amax(2).t()
    s = s.double()
    ds = far / 448 + 2 * U * top / 448
    assert ((s - top / 448).abs() <= ds * 1.001 + 2.0 ** -126).all()
    wide = s.t().repeat_interleave(128, 1)[:, :n]
    ds = ds.t().repeat_interleave(128, 1)[:, :n]
    bound = v.abs() * (F8_ROUND + 4 * U) * 1.001 + F8_TINY * wide * 1.001 + dv * 1.1 + 448 * ds * F8_ROUND
    assert ((q.double() * wide - v).abs() <= bound).all()


@pytest.mark.parametrize("m,n,k", PRODUCTS)
def test_product(m, n, k):
    data = operands(m, n, k, m + n)
    check_half(w.f8_gemm(*data), *product(*data))


@pytest.mark.parametrize("m,n,k", GATED)
def test_gated(m, n, k):
    data = operands(m, n, k, m + n, 2)
    for kind in ("silu", "gelu_tanh"):
        v, dv = gated(*data, kind)
        check_half(w.f8_gemm_gated(*data, kind, quantize=False), v, dv)
        check_codes(*w.f8_gemm_gated(*data, kind), v, dv)
        del v, dv


@pytest.mark.parametrize("m,n,k", [(9 * 2 ** 20, 130, 256), (300, 9 * 2 ** 20, 256), (40, 9 * 2 ** 20, 256), (32, 2 ** 27, 16)])
def test_offsets_beyond_31_bits(m, n, k):
    """x, the weights or the output larger than 2^31 bytes: the first and last rows and columns, and some between."""
    g = rng(n)
    xq = torch.randint(0, 256, (m, k), device="cuda", generator=g, dtype=torch.uint8) & 0x77
    wq = torch.randint(0, 256, (n, k), device="cuda", generator=g, dtype=torch.uint8) & 0x77
    xq, wq = xq.view(F8), wq.view(F8)
    sx = torch.rand(-(-k // 128), m, device="cuda", generator=g) * 2.0 ** -8
    sw = torch.rand(-(-n // 128), -(-k // 128), device="cuda", generator=g) * 2.0 ** -8

    def ends(total, block):
        """A few whole blocks of the rows: first, last, about 2^31 bytes into x or w or y, others."""
        at = {0, (total - 1) // block, 2 ** 31 // k // block, 2 ** 31 // 2 // max(1, min(m, n)) // block, total // 3 // block}
        return torch.cat([torch.arange(b * block, min(total, (b + 1) * block), device="cuda")
                          for b in sorted(at) if b * block < total])

    rows, cols = ends(m, 128), ends(n, 128)
    blocks = torch.unique(cols // 128)
    pick = (xq.view(torch.uint8)[rows].view(F8), sx[:, rows].contiguous(), wq.view(torch.uint8)[cols].view(F8), sw[blocks])
    v, dv = product(*pick)
    y = w.f8_gemm(xq, sx, wq, sw)
    check_half(y[rows][:, cols], v, dv)
    del y
    act, dact = gated(*pick, *pick[2:], "silu")
    q, s = w.f8_gemm_gated(xq, sx, wq, sw, wq, sw)
    q = q.view(torch.uint8)[rows][:, cols].view(F8)
    check_codes(q, s[blocks][:, rows], act, dact)


def test_long_k():
    """K at 2^20: many blocks, and one token's scales far apart."""
    for m, n in ((1, 40), (33, 130), (130, 70)):
        data = operands(m, n, 2 ** 20, m)
        check_half(w.f8_gemm(*data), *product(*data))


# sizes whose workgroups meet in the workspace: K in four, K in two, two workgroups a scale, K in parts
MEET = [(5, 500, 8208, False), (17, 1000, 8320, False), (3, 1030, 1040, True), (33, 8250, 272, True),
        (300, 200, 4112, False), (130, 300, 4112, True)]


def run(data, is_gated, ws, out=None):
    if is_gated:
        q, s = w.f8_gemm_gated(*data, workspace=ws)
        return torch.cat((q.view(torch.uint8).flatten(), s.view(torch.uint8).flatten()))
    return w.f8_gemm(*data, workspace=ws).view(torch.uint8).flatten()


def needs(m, n, k, is_gated):
    size = w.f8_gemm_gated_workspace_size(m, n, k) if is_gated else w.f8_gemm_workspace_size(m, n, k)
    assert size > 0
    return size


def test_one_workspace_for_all_whatever_it_holds():
    """Calls of different sizes in turn over one workspace that began with anything in it, and longer than asked."""
    ws = torch.empty(max(needs(*c) for c in MEET) + 512, dtype=torch.uint8, device="cuda")
    sets = [operands(m, n, k, i, 2 if g else 1) for i, (m, n, k, g) in enumerate(MEET)]
    want = [run(d, c[3], None) for d, c in zip(sets, MEET)]
    for fill in (0, 255, 1, None):
        if fill is None:
            ws.random_(0, 256)
        else:
            ws.fill_(fill)
        for i in (0, 2, 5, 1, 4, 3, 3, 4, 0, 5, 2, 2, 1):
            assert torch.equal(run(sets[i], MEET[i][3], ws), want[i])
    # no byte behind what was asked for is touched
    for d, c in zip(sets, MEET):
        need = needs(*c)
        ws.fill_(93)
        run(d, c[3], ws[:need])
        assert (ws[need:] == 93).all()


def test_two_graphs_over_one_workspace():
    """Captured one after the other over the same workspace, replayed in every order with eager calls between."""
    ws = torch.empty(max(needs(*c) for c in MEET), dtype=torch.uint8, device="cuda").random_(0, 256)
    sets = [operands(m, n, k, 50 + i, 2 if g else 1) for i, (m, n, k, g) in enumerate(MEET)]
    want = [run(d, c[3], None) for d, c in zip(sets, MEET)]
    graphs = []
    for i, (d, c) in enumerate(zip(sets, MEET)):
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            run(d, c[3], ws)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = run(d, c[3], ws), run(d, c[3], ws)
        graphs.append((graph, out))
    for turn in range(6):
        for i in (0, 1, 5, 2, 4, 3, 3, 1, 4, 0, 5, 0, 2):
            graphs[i][0].replay()
            if turn % 2:
                assert torch.equal(run(sets[5 - i], MEET[5 - i][3], ws), want[5 - i])
            if turn == 5:
                ws.random_(0, 256)                         # between calls it may hold anything
        for i in range(len(MEET)):
            graphs[i][0].replay()
            torch.cuda.synchronize()
            for out in graphs[i][1]:
                assert torch.equal(out, want[i])
                out.zero_()


def test_two_streams_at_once():
    """Each stream with a workspace of its own, their calls overlapping."""
    sets = [operands(m, n, k, 90 + i, 2 if g else 1) for i, (m, n, k, g) in enumerate(MEET)]
    want = [run(d, c[3], None) for d, c in zip(sets, MEET)]
    streams = [torch.cuda.Stream() for _ in MEET]
    spaces = [torch.empty(needs(*c), dtype=torch.uint8, device="cuda").random_(0, 256) for c in MEET]
    got = [[] for _ in MEET]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(run(sets[i], MEET[i][3], spaces[i]))
    torch.cuda.synchronize()
    for outs, v in zip(got, want):
        assert all(torch.equal(o, v) for o in outs)


@pytest.mark.parametrize("m,k,inner", [(1, 256, 1040), (7, 1024, 700 // 16 * 16), (64, 512, 8256), (150, 640, 1300 // 16 * 16),
                                       (2058, 1040, 7696)])
def test_feed_forward_block(m, k, inner):
    """norm, the gated product and the down product in a row, each against its definition in 64 bits from what
    the step before gave, and the whole within the quantisers' steps of the block in 64 bits."""
    g = rng(m)

    def weight(n, k):
        return (torch.randn(n, k, device="cuda", generator=g) / math.sqrt(k)).half()

    x = torch.randn(m, k, device="cuda", generator=g).half()
    res = torch.randn(m, k, device="cuda", generator=g).half()
    gain = (1 + 0.1 * torch.randn(k, device="cuda", generator=g)).half()
    halves = weight(inner, k), weight(inner, k), weight(k, inner)
    wg, wu, wd = (w.quantize_weight_f8(t) for t in halves)
    xq, xs, h = w.rmsnorm_quant(w.Mode.F8, x, gain, 1e-6, residual=res)
    aq, sa = w.f8_gemm_gated(xq, xs, *wg, *wu)
    y = w.f8_gemm(aq, sa, *wd)
    # the norm: K / 64 + 28 fp32 roundings of the sum, halved by the root, then the root, quotient and products
    s = x.double() + res.double()
    assert ((h.double() - s).abs() <= s.abs() * HALF_ROUND * 1.001 + HALF_TINY).all()
    v = s / (s.square().mean(1, keepdim=True) + 1e-6).sqrt() * gain.double()
    check_codes(xq, xs, v, ((k / 64 + 28) / 2 + 8) * U * v.abs())
    check_codes(aq, sa, *gated(xq, xs, *wg, *wu, "silu"))
    check_half(y, *product(aq, sa, *wd))
    # the whole: e4m3 rounds an operand to a relative 2^-3 / 12^(1/2) = 0.036 rms at most (0.025 over a
    # binade), six times on the way (x and a weight in the gate and in the up product, where the activation
    # keeps the size of an error; its result; the down weights), independent: 6^(1/2) 0.036 = 0.09 at most
    a = activation(v @ halves[0].double().t().contiguous(), "silu") * (v @ halves[1].double().t().contiguous())
    plain = a @ halves[2].double().t().contiguous()
    assert (y.double() - plain).square().mean().sqrt() <= 0.1 * plain.square().mean().sqrt()
    # the same from one captured step, replayed on other tokens
    static = [t.clone() for t in (x, res)]
    ws = w.f8_gemm_workspace(m, k, inner), w.f8_gemm_gated_workspace(m, inner, k)

    def step():
        q, s, h = w.rmsnorm_quant(w.Mode.F8, static[0], gain, 1e-6, residual=static[1])
        return h, w.f8_gemm(*w.f8_gemm_gated(q, s, *wg, *wu, workspace=ws[1]), *wd, workspace=ws[0])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gh, gy = step()
    for turn in range(3):
        static[0].copy_(x if turn != 1 else res)
        static[1].copy_(res if turn != 1 else x)           # the sum is the same
        gy.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(gh, h) and torch.equal(gy, y)

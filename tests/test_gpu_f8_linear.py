"""linear(Mode.F8) and linear_noalloc(Mode.F8) where the product meets in the workspace, with workspaces of
exactly what the call needs, and prompts whose products need none."""
import pytest

torch = pytest.importorskip("torch")

import w4a8_int8_gemm_amd as w  # noqa: E402

pytestmark = pytest.mark.gpu


def layer(m, n, k, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(m, k, device="cuda", generator=g).half()
    return x, *w.quantize_weight_f8((torch.randn(n, k, device="cuda", generator=g) * k ** -0.5).half())


def own_need(m, n, k):
    def up(v):
        return -(-v // 256) * 256
    return up(m * k) + up(4 * m * -(-k // 128)) + w.f8_gemm_workspace_size(m, n, k)


# K over workgroups in four, in two, in parts above 64 tokens; and products that need nothing
SIZES = [(5, 500, 8208, True), (17, 1000, 8320, True), (300, 200, 4112, True), (3, 700, 1040, False), (517, 2050, 2064, False)]


@pytest.mark.parametrize("m,n,k,meets", SIZES)
def test_exact_workspaces(m, n, k, meets):
    """Whatever the workspace held, not a byte behind it written, the bits of the quantizer and the product."""
    assert (w.f8_gemm_workspace_size(m, n, k) > 0) == meets
    x, wq, sw = layer(m, n, k, m)
    want = w.f8_gemm(*w.quantize_act_f8(x), wq, sw)
    need = own_need(m, n, k)
    ws = torch.empty(need + 4096, dtype=torch.uint8, device="cuda")
    for fill in (0, 255, None, None):
        ws.random_(0, 256) if fill is None else ws.fill_(fill)
        ws[need:] = 93
        assert torch.equal(w.linear(w.Mode.F8, x, wq, sw, workspace=ws[:need]), want)
        assert (ws[need:] == 93).all()
    assert torch.equal(w.linear(w.Mode.F8, x, wq, sw), want)
    full = torch.empty(w.linear_workspace_size(w.Mode.F8, m, k), dtype=torch.uint8, device="cuda").random_(0, 256)
    assert torch.equal(w.linear(w.Mode.F8, x, wq, sw, workspace=full), want)


def test_the_static_array_between_the_modes():
    """Every mode's calls in turn over the one array: what one leaves there is no matter to the next."""
    sets = [layer(m, n, k, m) for m, n, k, _ in SIZES]
    want = [w.f8_gemm(*w.quantize_act_f8(x), wq, sw) for x, wq, sw in sets]
    g = torch.Generator(device="cuda").manual_seed(9)
    others = []
    for m, k in ((40, 8192), (700, 4096), (9, 1024)):
        x = torch.randn(m, k, device="cuda", generator=g).half()
        wt = (torch.randn(96, k, device="cuda", generator=g) * 0.02).half()
        for mode, gs, (q, s) in ((w.Mode.W8A8_PC, 0, w.quantize_weight_int8(wt, 0)), (w.Mode.W4A8, 128, w.pack_weight_int4(wt, 128))):
            others.append((mode, x, q, s, gs, w.linear(mode, x, q, s, gs)))
    for turn in range(3):
        for i in range(len(sets)):
            assert torch.equal(w.linear_noalloc(w.Mode.F8, *sets[i]), want[i])
            mode, x, q, s, gs, y = others[(i + turn) % len(others)]
            assert torch.equal(w.linear_noalloc(mode, x, q, s, gs), y)


def test_the_static_array_in_a_graph():
    """Captured calls of both kinds, replayed with eager calls between that leave other bytes in the array."""
    sets = [layer(m, n, k, 30 + m) for m, n, k, _ in SIZES[:3]]
    want = [w.f8_gemm(*w.quantize_act_f8(x), wq, sw) for x, wq, sw in sets]
    big = layer(600, 130, 4096, 1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for s in sets:
            w.linear_noalloc(w.Mode.F8, *s)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = [w.linear_noalloc(w.Mode.F8, *s) for s in sets]
    for _ in range(4):
        for y in out:
            y.zero_()
        w.linear_noalloc(w.Mode.F8, *big)
        graph.replay()
        w.linear_noalloc(w.Mode.F8, *sets[2])
        torch.cuda.synchronize()
        for y, v in zip(out, want):
            assert torch.equal(y, v)


def test_prompts_that_fit_the_static_array():
    """57 and 51 MB of codes and scales, whose products need nothing of the workspace."""
    for m, n, k in ((4516, 4096, 12288), (4096, 2048, 12288)):
        assert w.f8_gemm_workspace_size(m, n, k) == 0
        x, wq, sw = layer(m, n, k, n)
        want = w.f8_gemm(*w.quantize_act_f8(x), wq, sw)
        assert torch.equal(w.linear_noalloc(w.Mode.F8, x, wq, sw), want)
        ws = torch.empty(own_need(m, n, k), dtype=torch.uint8, device="cuda")
        assert torch.equal(w.linear(w.Mode.F8, x, wq, sw, workspace=ws), want)

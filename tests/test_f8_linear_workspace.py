"""What linear(Mode.F8) and linear_noalloc(Mode.F8) ask of their workspace: the need of the call's own
columns, not the most of any."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import w4a8_int8_gemm_amd as w  # noqa: E402
from w4a8_int8_gemm_amd import ops  # noqa: E402

P = ctypes.c_void_p
X, W, SW, Y, WS = (P(4096 * i) for i in range(1, 6))
REFUSED = int(w.Status.ERR_WORKSPACE)


@pytest.fixture(scope="module")
def no_device():
    """Calls that are not refused end at the check of the device; with one they would run on these addresses."""
    if torch.cuda.is_available():
        pytest.skip("only without a GPU")


def own_need(m, n, k):
    def up(v):
        return -(-v // 256) * 256
    return up(m * k) + up(4 * m * -(-k // 128)) + w.f8_gemm_workspace_size(m, n, k)


# a product that meets in the workspace, by tokens, and products that need none there
SIZES = [(5, 500, 8208), (17, 1000, 8320), (300, 200, 4112), (1, 4096, 12288), (517, 4096, 4096), (4516, 4096, 12288)]


@pytest.mark.parametrize("m,n,k", SIZES)
def test_linear_takes_what_its_columns_need(no_device, m, n, k):
    L, need = w.lib(), own_need(m, n, k)
    assert need <= w.linear_workspace_size(w.Mode.F8, m, k)
    assert L.linear(3, X, m, k, W, SW, 0, n, Y, WS, need - 1, None) == REFUSED
    assert L.linear(3, X, m, k, W, SW, 0, n, Y, WS, need, None) == int(w.Status.ERR_DEVICE)


@pytest.mark.parametrize("m,n,k", [(4516, 4096, 12288), (8192, 6144, 6144), (4096, 4096, 12288), (3000, 4096, 16368)])
def test_noalloc_takes_what_fits_its_array(no_device, m, n, k):
    """Codes and scales below 64 MiB whose product needs nothing."""
    assert w.f8_gemm_workspace_size(m, n, k) == 0
    assert own_need(m, n, k) <= 1 << 26 < w.linear_workspace_size(w.Mode.F8, m, k)
    assert w.lib().linear_noalloc(3, X, m, k, W, SW, 0, n, Y, None) == int(w.Status.ERR_DEVICE)


def test_noalloc_refuses_what_does_not_fit(no_device):
    m, n, k = 4516, 200, 12288                             # few columns: K in parts, whose sums do not fit
    assert own_need(m, 4096, k) <= 1 << 26 < own_need(m, n, k)
    assert w.lib().linear_noalloc(3, X, m, k, W, SW, 0, n, Y, None) == REFUSED
    m = 5000
    assert own_need(m, 4096, 16368) > 1 << 26
    assert w.lib().linear_noalloc(3, X, m, 16368, W, SW, 0, 4096, Y, None) == REFUSED
    assert "workspace" in w.lib().w4a8_last_error().decode()


def test_wrapper(monkeypatch):
    """The wrapper refuses what the library would, and takes what it takes."""
    monkeypatch.setattr(ops, "_DEVICE_TYPE", "cpu")
    calls = []
    monkeypatch.setattr(ops, "_call", lambda index, fn, *args: calls.append(args))
    m, k = 300, 4112
    for n, parts in ((200, True), (16000, False)):
        need = own_need(m, n, k)
        assert (w.f8_gemm_workspace_size(m, n, k) > 0) == parts
        x = torch.zeros(m, k, dtype=torch.float16)
        wq, sw = torch.zeros(n, k, dtype=torch.uint8).view(torch.float8_e4m3fn), torch.ones(-(-n // 128), -(-k // 128))
        with pytest.raises(ValueError, match=f"workspace.*{need}"):
            w.linear(w.Mode.F8, x, wq, sw, workspace=torch.zeros(need - 1, dtype=torch.uint8))
        assert not calls
        w.linear(w.Mode.F8, x, wq, sw, workspace=torch.zeros(need, dtype=torch.uint8))
        w.linear(w.Mode.F8, x, wq, sw)
        assert [a[-1] for a in calls] == [need, need]
        calls.clear()

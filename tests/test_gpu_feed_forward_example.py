"""The feed-forward block's example: it runs, and its captured step gives what its calls give."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("feed_forward_block", os.path.join(ROOT, "examples", "feed_forward_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_main_runs(monkeypatch, capsys):
    monkeypatch.setattr("sys.argv", ["x", "--hidden", "512", "--inner", "1040", "--tokens", "300", "--steps", "3", "--batch", "2"])
    example().main()
    out = capsys.readouterr().out
    assert "prompt: 300 tokens" in out and "step: 2 tokens" in out


@pytest.mark.parametrize("tokens", [1, 40])
def test_steps_are_the_calls(tokens):
    """Two captured steps of two blocks, replayed in turn with new tokens each."""
    ex = example()
    blocks = [ex.FeedForwardBlock(256, 1040, "gelu_tanh", seed=i) for i in range(2)]
    steps = [ex.Step(b, tokens) for b in blocks]
    g = torch.Generator(device="cuda").manual_seed(2)
    for _ in range(4):
        for block, step in zip(blocks, steps):
            x, attention = (torch.randn(tokens, 256, device="cuda", generator=g).half() for _ in range(2))
            step.x.copy_(x)
            step.attention.copy_(attention)
            got = step()
            want = block(x, attention)
            torch.cuda.synchronize()
            for a, b in zip(got, want):
                assert torch.equal(a, b) and torch.isfinite(a).all()

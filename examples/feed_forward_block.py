"""The gated feed-forward block of a decoder layer in 8-bit floating point, from
the attention's output to the next layer's input:

    h = x + attention
    q = e4m3(norm(h))  ->  e4m3(act(q . gate^T) * (q . up^T))  ->  . down^T

The residual's addition, the norm and the quantization are one kernel, both
first products, the activation, their product and its quantization another.  A
prompt goes through as it is; single steps are captured once and replayed, with
weights and workspaces that are laid out before.  The weights are random.

    python examples/feed_forward_block.py [--tokens 4096] [--steps 100] [--batch 1]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import w4a8_int8_gemm_amd as w  # noqa: E402


class FeedForwardBlock:
    """One layer's norm, gate, up and down."""

    def __init__(self, hidden: int = 4096, inner: int = 12288, activation: str = "silu", eps: float = 1e-6, seed: int = 0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def weight(n, k):
            return w.quantize_weight_f8((torch.randn(n, k, device="cuda", generator=g) * k ** -0.5).half())

        self.hidden, self.inner, self.activation, self.eps = hidden, inner, activation, eps
        self.gate, self.up, self.down = weight(inner, hidden), weight(inner, hidden), weight(hidden, inner)
        self.gain = (1 + 0.1 * torch.randn(hidden, device="cuda", generator=g)).half()

    def workspaces(self, tokens):
        """What calls of so many tokens need, for one stream."""
        return (w.f8_gemm_gated_workspace(tokens, self.inner, self.hidden),
                w.f8_gemm_workspace(tokens, self.hidden, self.inner))

    def __call__(self, x, attention, workspaces=(None, None)):
        """x, attention fp16 [T, hidden]: (the residual stream behind the attention, the block's output, which
        the next layer's norm adds to it)."""
        q, s, h = w.rmsnorm_quant(w.Mode.F8, x, self.gain, self.eps, residual=attention)
        a, sa = w.f8_gemm_gated(q, s, *self.gate, *self.up, self.activation, workspace=workspaces[0])
        return h, w.f8_gemm(a, sa, *self.down, workspace=workspaces[1])


class Step:
    """A block's step for a fixed number of tokens, captured once: write x and attention, call, read h and y."""

    def __init__(self, block, tokens):
        self.x = torch.zeros(tokens, block.hidden, dtype=torch.float16, device="cuda")
        self.attention = torch.zeros_like(self.x)
        self.workspaces = block.workspaces(tokens)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            block(self.x, self.attention, self.workspaces)
        torch.cuda.current_stream().wait_stream(side)
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self.h, self.y = block(self.x, self.attention, self.workspaces)

    def __call__(self):
        self.graph.replay()
        return self.h, self.y


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--inner", type=int, default=12288)
    ap.add_argument("--tokens", type=int, default=4096, help="of the prompt")
    ap.add_argument("--steps", type=int, default=100, help="single steps after it")
    ap.add_argument("--batch", type=int, default=1, help="tokens of a step")
    a = ap.parse_args()
    block = FeedForwardBlock(a.hidden, a.inner)
    g = torch.Generator(device="cuda").manual_seed(1)

    def rows(n):
        return torch.randn(n, a.hidden, device="cuda", generator=g).half()

    def timed(fn, n):
        begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        begin.record()
        for _ in range(n):
            out = fn()
        end.record()
        end.synchronize()
        return out, begin.elapsed_time(end) / n * 1000

    x, attention = rows(a.tokens), rows(a.tokens)
    block(x, attention)                                  # warm-up
    (h, y), us = timed(lambda: block(x, attention), 3)
    print(f"prompt: {a.tokens} tokens, {us:.1f} us, |y| {float(y.float().norm()):.4f}")
    step = Step(block, a.batch)
    step.x.copy_(x[-a.batch:])
    step.attention.copy_(attention[-a.batch:])
    step()
    (h, y), us = timed(step, a.steps)
    print(f"step: {a.batch} tokens, {us:.1f} us, |y| {float(y.float().norm()):.4f}")


if __name__ == "__main__":
    main()

"""The attention block of a decoder layer in the library's number formats, from
its normalised input to its output product:

    qkv = linear(x)  ->  rotary_axes  ->  kv4_write  ->  kv4_attention  ->  linear

A prompt goes through in one call, then tokens one at a time, as a serving
loop would do it: the cache, its page table and the workspaces are kept, the
sequences' lengths advance on the device.  The linear layers are W4A8, the
cache is 4-bit; the weights are random.

    python examples/attention_block.py [--tokens 1000] [--steps 8] [--sequences 3]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import w4a8_int8_gemm_amd as w  # noqa: E402


class AttentionBlock:
    """One layer's attention for a fixed set of sequences."""

    def __init__(self, sequences: int, longest: int, hidden: int = 4096, q_heads: int = 32, kv_heads: int = 8,
                 head_dim: int = 128, sections=(24, 20, 20), page_size: int = 64, group_size: int = 64, seed: int = 0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.q_heads, self.kv_heads, self.head_dim, self.sections = q_heads, kv_heads, head_dim, sections

        def weight(n, k):
            return w.pack_weight_int4((torch.randn(n, k, device="cuda", generator=g) * 0.02).half(), 128)

        self.qkv = weight((q_heads + 2 * kv_heads) * head_dim, hidden)
        self.out = weight(hidden, q_heads * head_dim)
        half = sum(sections)
        self.inv_freq = (1e6 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)).float()
        # pages dealt out once, in a mixed order
        per = -(-longest // page_size)
        self.cache = w.KV4Cache.empty(sequences * per, kv_heads, page_size, head_dim, group_size)
        self.page_table = torch.randperm(sequences * per, device="cuda", generator=g).to(torch.int32).view(sequences, per)
        self.lens = torch.zeros(sequences, dtype=torch.int32, device="cuda")

    def __call__(self, x, positions, counts):
        """x fp16 [T, hidden]: counts[b] new tokens of each sequence, in order; positions int64 [axes, T]."""
        T, D, page = x.shape[0], self.head_dim, self.cache.page_size
        q_heads, kv_heads = self.q_heads, self.kv_heads
        # where the new tokens go
        new = torch.tensor(counts, dtype=torch.int32).to(x.device)
        starts = torch.nn.functional.pad(new.cumsum(0), (1, 0)).to(torch.int32)
        seq = torch.repeat_interleave(torch.arange(len(counts), device=x.device), new, output_size=T)
        at = self.lens[seq].long() + torch.arange(T, device=x.device) - starts[seq].long()
        slots = self.page_table[seq, at // page].long() * page + at % page
        self.lens += new

        qkv = w.linear(w.Mode.W4A8, x, *self.qkv, 128).view(T, q_heads + 2 * kv_heads, D)
        qk = w.rotary_axes(qkv[:, :q_heads + kv_heads], positions, self.inv_freq, self.sections, interleaved=True)
        w.kv4_write(qk[:, q_heads:], qkv[:, q_heads + kv_heads:], slots, self.cache)
        o = w.kv4_attention(qk[:, :q_heads], self.cache, self.page_table, self.lens, q_starts=starts,
                            max_q=max(counts))
        return w.linear(w.Mode.W4A8, o.view(T, q_heads * D), *self.out, 128)


def text_positions(first, counts, device="cuda"):
    """Text has the same position on every axis."""
    p = torch.cat([torch.arange(f, f + n) for f, n in zip(first, counts)])
    return p.expand(3, -1).contiguous().to(device)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=1000, help="longest prompt")
    ap.add_argument("--steps", type=int, default=8, help="tokens generated after it")
    ap.add_argument("--sequences", type=int, default=3)
    a = ap.parse_args()
    counts = [max(1, a.tokens - 37 * b) for b in range(a.sequences)]
    block = AttentionBlock(a.sequences, a.tokens + a.steps)
    g = torch.Generator(device="cuda").manual_seed(1)

    def run(first, counts):
        x = torch.randn(sum(counts), 4096, device="cuda", generator=g).half()
        begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        positions = text_positions(first, counts)
        begin.record()
        y = block(x, positions, counts)
        end.record()
        end.synchronize()
        return y, begin.elapsed_time(end)

    run([0] * a.sequences, counts)                       # warm-up on the same pages
    block.lens.zero_()
    y, ms = run([0] * a.sequences, counts)
    print(f"prompt: {sum(counts)} tokens of {a.sequences} sequences, {ms:.3f} ms, output {tuple(y.shape)}")
    for s in range(a.steps):
        y, ms = run([n + s for n in counts], [1] * a.sequences)
        print(f"token {s}: {ms:.3f} ms, |y| {float(y.float().norm()):.4f}")


if __name__ == "__main__":
    main()

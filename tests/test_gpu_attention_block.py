"""The attention block's operators together with the linear layers, as the example runs them."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")

import w4a8_int8_gemm_amd as w  # noqa: E402

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("attention_block", os.path.join(ROOT, "examples", "attention_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def plain_rotary(x, positions, inv_freq, sections):
    half = inv_freq.numel()
    i = torch.arange(half, device=x.device)
    left = i // 3 < torch.tensor(sections, device=x.device)[i % 3]
    axis = torch.where(left, i % 3, torch.zeros_like(i))
    a = positions[axis].t().double() * inv_freq.double()
    c, s = a.cos()[:, None], a.sin()[:, None]
    p, q = x.double()[..., :half], x.double()[..., half:]
    return torch.cat((p * c - q * s, q * c + p * s), -1)


def test_prompt_then_tokens():
    """Every call's output against the same steps with rotary positions and attention in 64 bits
    (the linear layers and the cache's codes are the library's on both sides)."""
    ex = example()
    hidden, hq, hk, D = 512, 4, 2, 128
    block = ex.AttentionBlock(2, 90, hidden, hq, hk, D, page_size=16, group_size=64)
    seen = [0, 0]
    g = torch.Generator(device="cuda").manual_seed(3)
    for counts in ([70, 33], [1, 1], [1, 5], [1, 1]):
        x = torch.randn(sum(counts), hidden, device="cuda", generator=g).half()
        pos = ex.text_positions(seen, counts)
        y = block(x, pos, counts)
        seen = [n + c for n, c in zip(seen, counts)]
        assert block.lens.tolist() == seen
        qkv = w.linear(w.Mode.W4A8, x, *block.qkv, 128).view(-1, hq + 2 * hk, D)
        q = plain_rotary(qkv[:, :hq], pos, block.inv_freq, block.sections)
        rows, first = [], 0
        for b, m in enumerate(counts):
            n = seen[b]
            j = torch.arange(n, device="cuda")
            slots = block.page_table[b].long()[j // 16] * 16 + j % 16
            k, v = (t.double() for t in w.kv4_read(block.cache, slots))
            s = torch.matmul(q[first:first + m].transpose(0, 1), k.repeat_interleave(hq // hk, 1).permute(1, 2, 0).contiguous())
            s = s * D ** -0.5
            hide = j[None] > torch.arange(n - m, n, device="cuda")[:, None]
            p = s.masked_fill(hide, float("-inf")).softmax(-1)
            rows.append(torch.matmul(p, v.repeat_interleave(hq // hk, 1).transpose(0, 1).contiguous()).transpose(0, 1))
            first += m
        o = torch.cat(rows).half().reshape(-1, hq * D)
        want = w.linear(w.Mode.W4A8, o, *block.out, 128).float()
        # the two o's differ by a few roundings to fp16 (of q, the read-back k and v, weights and o: 2^-11 each),
        # and int8 quantisation turns a difference at a border into a step, 1 / 127 of a row's largest value
        assert float((y.float() - want).norm() / want.norm()) < 8 * 2.0 ** -11 + 1 / 127


def test_replaying_a_step_gives_the_same_output():
    ex = example()
    outs = []
    for _ in range(2):
        block = ex.AttentionBlock(3, 200, 512, 4, 2, 64, sections=(12, 10, 10), page_size=32, group_size=32, seed=5)
        g = torch.Generator(device="cuda").manual_seed(7)
        counts, seen, ys = [120, 1, 63], [0, 0, 0], []
        for _ in range(3):
            x = torch.randn(sum(counts), 512, device="cuda", generator=g).half()
            ys.append(block(x, ex.text_positions(seen, counts), counts))
            seen = [n + c for n, c in zip(seen, counts)]
            counts = [1, 1, 1]
        outs.append(ys)
    for a, b in zip(*outs):
        assert torch.equal(a, b)

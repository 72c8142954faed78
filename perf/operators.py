"""The operators of the attention block next to the int8 linear layer, as they are measured.

Four operators that a decoder layer needs between its qkv and its output product:

* ``rotary``: rotary positions with up to three axes (time, height, width) on
  the query and key heads of the qkv product's output;
* ``cache``: keys and values quantised to 4 bits as they are written into a
  paged cache, and the written tokens read back;
* ``read``: whole sequences read back from that cache;
* ``attention``: attention of one or many query tokens a sequence over the
  4-bit cache, with the log of the softmax sum.

The cache's format: pages [pages, kv_heads, page_size, head_dim / 2] of packed
codes for K and for V, with fp32 scales [pages, kv_heads, page_size,
head_dim / group].  A code is the symmetric int4 rule's: s = fl32(amax / 7),
q = round_half_away(fl32(x / s)) in [-7, 7], two's complement nibbles, the even
element low.  Within a row the bytes are stored transposed: K's row is
[head_dim / 32][4 words] stored as [4 words][head_dim / 32], V's row is
[head_dim / 32][16 bytes] stored as [16 bytes][head_dim / 32].
"""
from __future__ import annotations

import math

import torch

own = False

DEVICE = "cuda"


# --------------------------------------------------------------------------- cases

def _rotary(name, tokens, q_heads, kv_heads, head_dim, rotary_dim, axes, s1, s2, interleaved):
    return dict(name=name, op="rotary", tokens=tokens, q_heads=q_heads, kv_heads=kv_heads, head_dim=head_dim,
                rotary_dim=rotary_dim, axes=axes, height=s1, width=s2, interleaved=interleaved)


def _cache(name, op, tokens, kv_heads, head_dim, group, page):
    return dict(name=name, op=op, tokens=tokens, kv_heads=kv_heads, head_dim=head_dim, group=group, page=page)


def _attention(name, sequences, longest, shortest, q_longest, q_shortest, q_heads, kv_heads, head_dim, group, page,
               causal=True, window=0):
    return dict(name=name, op="attention", sequences=sequences, longest=longest, shortest=shortest,
                q_longest=q_longest, q_shortest=q_shortest, q_heads=q_heads, kv_heads=kv_heads, head_dim=head_dim,
                group=group, page=page, causal=causal, window=window)


def listed():
    return [
        # one generated token of the 32 + 8 heads x 128 decoder layer: latency alone counts
        _rotary("rotary 1 token", 1, 32, 8, 128, 128, 3, 20, 20, True),
        # the 4516-token context of the W4A8 decoder layer, positions of text, images and video
        _rotary("rotary 4516 tokens", 4516, 32, 8, 128, 128, 3, 20, 20, True),
        # one step of 32 sequences: a new token each, written at scattered slots
        _cache("cache 32 tokens", "cache", 32, 8, 128, 128, 16),
        # the prompt of 4516 tokens written at once, scales for half heads
        _cache("cache 4516 tokens", "cache", 4516, 8, 128, 64, 64),
        # a short prefix read back (odd length, small heads, fine groups)
        _cache("read 517 tokens", "read", 517, 4, 64, 32, 16),
        # a long context taken out of the cache, to move it or to recompute from it
        _cache("read 65533 tokens", "read", 65533, 8, 128, 32, 128),
        # one sequence, one new token, short context: latency alone counts
        _attention("decode 1 x 517", 1, 517, 517, 1, 1, 32, 8, 128, 128, 16),
        # a serving batch: 32 sequences of uneven lengths up to the 4516-token context
        _attention("decode 32 x <= 4516", 32, 4516, 129, 1, 1, 32, 8, 128, 128, 16),
        # one very long sequence: its keys split over the whole chip
        _attention("decode 1 x 131075", 1, 131075, 131075, 1, 1, 32, 8, 128, 64, 64),
        # a few drafted tokens a sequence checked at once, own keys per head, sliding window
        _attention("verify 8 x 5, window", 8, 3001, 700, 5, 2, 16, 16, 64, 32, 32, window=1024),
        # the prompt itself: 4516 tokens, causal
        _attention("prefill 4516", 1, 4516, 4516, 4516, 4516, 32, 8, 128, 128, 16),
        # uneven chunks of prompts behind longer cached prefixes, next to a generated token
        _attention("chunks 4 x <= 1000", 4, 9000, 700, 1000, 1, 32, 8, 128, 64, 64),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def _head(rng):
    head_dim = rng.choice((64, 128, 128, 256))
    group = rng.choice([g for g in (32, 64, 128, 256) if g <= head_dim <= 4 * g])
    return head_dim, group


def draw(rng):
    op = rng.choice(("rotary", "cache", "read", "attention", "attention", "attention"))
    if op == "rotary":
        head_dim = rng.choice((64, 128, 256))
        rotary_dim = rng.choice((head_dim, head_dim, head_dim // 2))
        axes = rng.choice((1, 2, 3))
        most = rotary_dim // 2 // max(axes, 2)          # pairs that an axis behind the first may have
        s1 = rng.randint(1, most) if axes > 1 else 0
        s2 = rng.randint(1, most) if axes > 2 else 0
        kv = rng.choice((1, 2, 4, 8))
        case = _rotary("", _log(rng, 1, 8192), kv * rng.choice((1, 2, 4, 5, 8)), kv, head_dim, rotary_dim, axes,
                       s1, s2, rng.random() < 0.5)
    elif op in ("cache", "read"):
        head_dim, group = _head(rng)
        high = 8192 if op == "cache" else 65536
        case = _cache("", op, _log(rng, 1, high * 128 // head_dim // 2), rng.choice((1, 2, 3, 4, 8)), head_dim, group,
                      rng.choice((16, 32, 64, 128, 256)))
    else:
        head_dim, group = _head(rng)
        kv = rng.choice((1, 2, 4, 8))
        q_heads = kv * rng.choice((1, 2, 3, 4, 7, 8))
        kind = rng.choice(("decode", "decode", "verify", "prefill"))
        page = rng.choice((16, 32, 64, 128, 256))
        window = rng.choice((0, 0, 0, _log(rng, 16, 4096)))
        if kind == "decode":
            n = _log(rng, 1, 64)
            longest = _log(rng, 1, min(131072, 32 * 4516 * 8 * 128 // (n * kv * head_dim)))
            q_long, q_short = 1, 1
        elif kind == "verify":
            n, q_long = _log(rng, 1, 16), rng.randint(2, 16)
            longest = q_long + _log(rng, 1, 8192 * 128 // head_dim)
            q_short = rng.randint(1, q_long)
        else:
            n, q_long = rng.randint(1, 4), _log(rng, 17, 1500)
            longest = q_long + rng.choice((0, _log(rng, 1, 4096)))
            q_short = rng.randint(1, q_long)
        shortest = max(q_long, rng.randint(0, longest)) if q_long > 1 else rng.randint(0, longest)
        if n == 1:
            shortest, q_short = longest, q_long
        case = _attention("", n, longest, shortest, q_long, q_short, q_heads, kv, head_dim, group, page,
                          causal=rng.random() < 0.8, window=window)
        if not case["causal"]:
            case["window"] = 0
    case.pop("name")
    return case


# --------------------------------------------------------------------------- what a case holds

def _spread(longest, shortest, n):
    """n whole lengths from longest to shortest, in a fixed mixed order."""
    out = [longest - (longest - shortest) * i // max(1, n - 1) for i in range(n)]
    return out[1::2] + out[0::2]


def _lengths(case):
    n = case["sequences"]
    kv = _spread(case["longest"], case["shortest"], n)
    q = _spread(case["q_longest"], case["q_shortest"], n)
    return kv, q


def _visible(case):
    """(query, key) pairs inside the mask, and keys that some query of their sequence sees."""
    pairs = keys = 0
    for kv, q in zip(*_lengths(case)):
        if not case["causal"]:
            pairs, keys = pairs + q * kv, keys + kv
            continue
        w = case["window"] or kv
        lo = max(0, kv - q + 1 - w)
        keys += kv - lo
        # the query at position p sees min(p + 1, w) keys
        first, last = kv - q + 1, kv
        full = max(0, last - max(first, w) + 1)          # queries that see a whole window
        part = q - full
        pairs += full * w + (first + first + part - 1) * part // 2
    return pairs, keys


def work(case):
    d = case["head_dim"]
    if case["op"] == "rotary":
        heads, t = case["q_heads"] + case["kv_heads"], case["tokens"]
        # values in and out, positions; a rotated pair takes six operations
        return {"bytes": 4 * t * heads * d + 8 * t * case["axes"], "flops": 3 * t * heads * case["rotary_dim"]}
    packed = case["kv_heads"] * 2 * (d // 2 + 4 * (d // case["group"]))   # K's and V's bytes of a token in the cache
    plain = case["kv_heads"] * 2 * 2 * d                                   # and outside it
    if case["op"] == "cache":
        t = case["tokens"]                       # read plain, write packed; read packed, write plain
        return {"bytes": t * (2 * plain + 2 * packed + 8), "flops": t * case["kv_heads"] * 2 * d * 6}
    if case["op"] == "read":
        t = case["tokens"]
        return {"bytes": t * (plain + packed + 8), "flops": t * case["kv_heads"] * 2 * d}
    pairs, keys = _visible(case)
    q = sum(_lengths(case)[1])
    io = q * case["q_heads"] * (2 * d + 2 * d + 4)                         # queries, outputs, logs
    return {"bytes": keys * packed + io, "flops": 4 * d * case["q_heads"] * pairs}


# --------------------------------------------------------------------------- inputs

def _generator(seed):
    return torch.Generator(device=DEVICE).manual_seed(int(seed))


def _heads_of_qkv(tokens, q_heads, kv_heads, head_dim, g):
    """What the qkv product gives: q, k and v heads side by side in one row a token."""
    qkv = torch.randn(tokens, q_heads + 2 * kv_heads, head_dim, device=DEVICE, dtype=torch.float16, generator=g)
    return qkv, qkv[:, :q_heads], qkv[:, q_heads:q_heads + kv_heads], qkv[:, q_heads + kv_heads:]


def _outliers(k):
    """Keys have a few channels that are several times the others."""
    k[..., 3::29] *= 4
    return k


def _positions(tokens, axes, g):
    """Positions of a context of text and frames, in its later part (up to 10^6 tokens in)."""
    start = int(torch.randint(0, 1 << 20, (1,), device=DEVICE, generator=g))
    t = torch.arange(tokens, device=DEVICE, dtype=torch.int64)
    rows = [start + t // 7, start + (t // 37) % 41, start + t % 37]
    return torch.stack(rows[:axes]).contiguous()


def _nibbles(codes):
    """Codes [..., d] (int64 in [-7, 7]) to natural bytes [..., d / 2], the even element low."""
    u = codes & 15
    return (u[..., 0::2] | (u[..., 1::2] << 4)).to(torch.uint8)


def _codes(natural):
    """The inverse of _nibbles, in fp32."""
    u = torch.stack((natural & 15, natural >> 4), -1).flatten(-2).to(torch.float32)
    return u - 16.0 * (u >= 8)


def _stored(natural, unit):
    """Natural row bytes to the stored order: [d / 32][16 / unit units] transposed, units of `unit` bytes."""
    s = natural.shape
    return natural.reshape(*s[:-1], s[-1] // 16, 16 // unit, unit).transpose(-3, -2).reshape(s)


def _natural(stored, unit):
    s = stored.shape
    return stored.reshape(*s[:-1], 16 // unit, s[-1] // 16, unit).transpose(-3, -2).reshape(s)


K_UNIT, V_UNIT = 4, 1


def _quantise(x, group):
    """The int4 rule: (codes int64, scales fp32), the quotients rounded to 32 bits once."""
    g = x.to(torch.float32).unflatten(-1, (-1, group))
    s = (g.abs().amax(-1).double() / 7).float()
    t = torch.where(s[..., None] > 0, g.double() / s[..., None].double(), torch.zeros_like(g).double()).float()
    whole = torch.trunc(t)
    q = whole + torch.sign(t) * ((t - whole).abs() >= 0.5)
    return q.clamp(-7, 7).flatten(-2).to(torch.int64), s


def _dequantise(codes, scale, group):
    return (codes.unflatten(-1, (-1, group)) * scale[..., None]).flatten(-2)


def _empty_cache(pages, case):
    h, p, d = case["kv_heads"], case["page"], case["head_dim"]
    made = {}
    for n in ("k", "v"):
        made[n] = torch.zeros(pages, h, p, d // 2, device=DEVICE, dtype=torch.uint8)
        made[n + "_scale"] = torch.zeros(pages, h, p, d // case["group"], device=DEVICE, dtype=torch.float32)
    return made


def _handle(state):
    """The cache's handle, which a program makes once and keeps: it holds the four tensors as they are."""
    import w4a8_int8_gemm_amd as w
    return w.KV4Cache(state["k"], state["k_scale"], state["v"], state["v_scale"])


def prepare(case, seed):
    g = _generator(seed)
    state = dict(case)
    d = case["head_dim"]
    if case["op"] == "rotary":
        n = case["q_heads"] + case["kv_heads"]
        qkv, _, _, _ = _heads_of_qkv(case["tokens"], case["q_heads"], case["kv_heads"], d, g)
        r = case["rotary_dim"]
        state["x"] = qkv[:, :n]
        state["positions"] = _positions(case["tokens"], case["axes"], g)
        state["inv_freq"] = (1.0 / 1e6 ** (torch.arange(0, r, 2, device=DEVICE, dtype=torch.float64) / r)).float()
        rest = (case["height"], case["width"])[:case["axes"] - 1]
        state["sections"] = (r // 2 - sum(rest),) + tuple(rest)
        state["axis"] = _axis_of_pair(r // 2, state["sections"], case["interleaved"])
        return state
    if case["op"] in ("cache", "read"):
        t = case["tokens"]
        pages = -(-t // case["page"]) + 3
        state.update(_empty_cache(pages, case))
        if case["op"] == "cache":
            # scattered slots: every sequence's next token lies in a page of its own
            state["slots"] = torch.randperm(pages * case["page"], device=DEVICE, generator=g)[:t].contiguous()
            _, _, kk, vv = _heads_of_qkv(t, 4 * case["kv_heads"], case["kv_heads"], d, g)
            state["new_k"], state["new_v"] = _outliers(kk), vv
        else:
            order = torch.randperm(pages, device=DEVICE, generator=g)
            at = torch.arange(t, device=DEVICE)
            state["slots"] = (order[at // case["page"]] * case["page"] + at % case["page"]).contiguous()
            _fill(state, case, g)
    else:
        kv, q = _lengths(case)
        per = [-(-n // case["page"]) for n in kv]
        most = max(1, max(per))
        pages = sum(per) + 2
        state.update(_empty_cache(pages, case))
        _fill(state, case, g)
        order = torch.randperm(pages, device=DEVICE, generator=g).to(torch.int32)
        table = torch.zeros(len(kv), most, dtype=torch.int32, device=DEVICE)
        first = 0
        for b, n in enumerate(per):
            table[b, :n] = order[first:first + n]
            first += n
        state["page_table"] = table
        state["kv_lens"] = torch.tensor(kv, dtype=torch.int32, device=DEVICE)
        starts = [0]
        for n in q:
            starts.append(starts[-1] + n)
        state["q_starts"] = torch.tensor(starts, dtype=torch.int32, device=DEVICE)
        state["max_q"] = max(q)
        state["q"] = _heads_of_qkv(starts[-1], case["q_heads"], case["kv_heads"], d, g)[1]
        state["scale"] = d ** -0.5
    if own:
        # what a program keeps next to its cache: the handle and the workspace
        state["cache"] = _handle(state)
        if case["op"] == "attention":
            import w4a8_int8_gemm_amd as w
            state["workspace"] = w.kv4_attention_workspace(state["cache"], case["q_heads"], state["q"].shape[0],
                                                           case["sequences"], state["max_q"])
    return state


def _fill(state, case, g):
    """A cache full of quantised keys and values, in slices that keep the memory small."""
    pages, h, p, _ = state["k"].shape
    step = max(1, (1 << 25) // (h * p * case["head_dim"]))
    for n, unit in (("k", K_UNIT), ("v", V_UNIT)):
        for at in range(0, pages, step):
            m = min(step, pages - at)
            x = torch.randn(m, h, p, case["head_dim"], device=DEVICE, dtype=torch.float16, generator=g)
            codes, s = _quantise(_outliers(x) if n == "k" else x, case["group"])
            state[n][at:at + m] = _stored(_nibbles(codes), unit)
            state[n + "_scale"][at:at + m] = s


# --------------------------------------------------------------------------- one pass

def run(state):
    op = state["op"]
    if own:
        import w4a8_int8_gemm_amd as w
        if op == "rotary":
            return w.rotary_axes(state["x"], state["positions"], state["inv_freq"], state["sections"],
                                 state["interleaved"])
        if op == "cache":
            w.kv4_write(state["new_k"], state["new_v"], state["slots"], state["cache"])
            return w.kv4_read(state["cache"], state["slots"])
        if op == "read":
            return w.kv4_read(state["cache"], state["slots"])
        return w.kv4_attention(state["q"], state["cache"], state["page_table"], state["kv_lens"],
                               q_starts=state["q_starts"], max_q=state["max_q"], causal=state["causal"],
                               window=state["window"], scale=state["scale"], workspace=state["workspace"],
                               return_lse=True)
    if op == "rotary":
        return _plain_rotary(state)
    if op == "cache":
        _plain_write(state)
        return _plain_read(state)
    if op == "read":
        return _plain_read(state)
    return _plain_attention(state)


def _axis_of_pair(pairs, sections, interleaved):
    """Which axis turns each pair: runs of sections[a] pairs, or the axes in turn while each has pairs left."""
    i = torch.arange(pairs, device=DEVICE)
    ends = torch.cumsum(torch.tensor(sections, device=DEVICE), 0)
    if not interleaved:
        return (i[:, None] >= ends).sum(-1)
    n = len(sections)
    left = i // n < torch.tensor(sections, device=DEVICE)[i % n]
    return torch.where(left, i % n, torch.zeros_like(i))


def _plain_rotary(state):
    x, half = state["x"].float(), state["rotary_dim"] // 2
    # far positions: the angle in 64 bits, its cosine and sine rounded to 32
    angle = state["positions"][state["axis"]].t().double() * state["inv_freq"].double()
    c, s = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    a, b, rest = x[..., :half], x[..., half:2 * half], x[..., 2 * half:]
    return torch.cat((a * c - b * s, b * c + a * s, rest), -1).half()


def _plain_write(state):
    page, at = state["slots"] // state["page"], state["slots"] % state["page"]
    for n, x, unit in (("k", state["new_k"], K_UNIT), ("v", state["new_v"], V_UNIT)):
        codes, s = _quantise(x, state["group"])
        state[n][page, :, at] = _stored(_nibbles(codes), unit)
        state[n + "_scale"][page, :, at] = s


def _plain_read(state):
    page, at = state["slots"] // state["page"], state["slots"] % state["page"]

    def one(n, unit):
        codes = _codes(_natural(state[n][page, :, at], unit))
        return _dequantise(codes, state[n + "_scale"][page, :, at], state["group"]).half()

    return one("k", K_UNIT), one("v", V_UNIT)


def _plain_attention(state):
    table, lens, starts = state["page_table"].long(), state["kv_lens"].long(), state["q_starts"].long()
    n, hk, d = table.shape[0], state["kv_heads"], state["head_dim"]
    t, hq = state["q"].shape[:2]

    def cached(name, unit):                       # [n, hk, keys, d] in fp32
        codes = state[name][table].transpose(1, 2).flatten(2, 3)
        scale = state[name + "_scale"][table].transpose(1, 2).flatten(2, 3)
        return _dequantise(_codes(_natural(codes, unit)), scale, state["group"])

    k, v = cached("k", K_UNIT), cached("v", V_UNIT)
    keys = k.shape[2]
    # the ragged queries as [n, max_q], rows past a sequence's own left at zero
    m = state["max_q"]
    seq = torch.bucketize(torch.arange(t, device=DEVICE), starts[1:], right=True)
    row = torch.arange(t, device=DEVICE) - starts[seq]
    q = torch.zeros(n, m, hq, d, device=DEVICE)
    q[seq, row] = state["q"].float()
    q = q.reshape(n, m, hk, hq // hk, d).permute(0, 2, 3, 1, 4).reshape(n, hk, hq // hk * m, d)
    s = torch.matmul(q, k.transpose(-1, -2).contiguous()).reshape(n, hk, hq // hk, m, keys) * state["scale"]
    j = torch.arange(keys, device=DEVICE)
    seen = (j < lens[:, None])[:, None].expand(n, m, keys)
    if state["causal"]:
        # the last query stands at the last key
        pos = lens[:, None] - (starts[1:] - starts[:-1])[:, None] + torch.arange(m, device=DEVICE)
        seen = seen & (j <= pos[..., None])
        if state["window"]:
            seen = seen & (j > pos[..., None] - state["window"])
    seen = seen[:, None, None]
    s = torch.where(seen, s, torch.full_like(s, -math.inf))
    top = s.amax(-1, keepdim=True)
    safe = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    p = torch.exp(s - safe)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.reshape(n, hk, -1, keys), v).reshape(n, hk, hq // hk, m, d)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    lse = (safe + torch.log(total))[..., 0]
    o = o.permute(0, 3, 1, 2, 4).reshape(n, m, hq, d)[seq, row]
    lse = lse.permute(0, 3, 1, 2).reshape(n, m, hq)[seq, row]
    return o.half(), lse


# --------------------------------------------------------------------------- the same from the definitions, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"rotary": _exact_rotary, "cache": _exact_cache, "read": _exact_read,
            "attention": _exact_attention}[case["op"]](case, s)


def _exact_rotary(case, s):
    half, n, sections = case["rotary_dim"] // 2, case["axes"], s["sections"]
    axis = []
    if case["interleaved"]:
        for i in range(half):
            axis.append(i % n if i // n < sections[i % n] else 0)
    else:
        for a in range(n):
            axis += [a] * sections[a]
    x = s["x"].double()
    y = x.clone()
    for i in range(half):
        angle = (s["positions"][axis[i]].double() * s["inv_freq"][i].double())[:, None]
        z = torch.complex(x[..., i], x[..., i + half]) * torch.polar(torch.ones_like(angle), angle)
        y[..., i], y[..., i + half] = z.real, z.imag
    return y


def _exact_values(x, group):
    """What x stands for after the int4 rule; the rule's two roundings to 32 bits are part of its definition."""
    parts = []
    for at in range(0, x.shape[-1], group):
        p = x[..., at:at + group].double()
        top = torch.linalg.vector_norm(p, ord=math.inf, dim=-1, keepdim=True)
        s = (top / 7).float().double()
        t = (p / torch.where(s > 0, s, torch.ones_like(s))).float().double()
        q = torch.copysign(torch.floor(t.abs() + 0.5), t)
        parts.append(torch.clamp(q, -7, 7) * s)
    return torch.cat(parts, -1)


def _exact_cache(case, s):
    return _exact_values(s["new_k"], case["group"]), _exact_values(s["new_v"], case["group"])


def _exact_gather(case, s, name, page, at, head=None):
    """Values of the tokens at (page, at): every element's byte by its place, K and V apart."""
    d, n = case["head_dim"], case["head_dim"] // 32
    e = torch.arange(d, device=DEVICE)
    block, inside = e // 32, e % 32 // 2
    byte = ((inside // 4) * n + block) * 4 + inside % 4 if name == "k" else inside * n + block
    pick = (lambda x: x[page, :, at]) if head is None else (lambda x: x[page, head, at])
    raw = pick(s[name])[..., byte].int()
    code = torch.where(e % 2 == 0, raw % 16, raw // 16)
    code = torch.where(code > 7, code - 16, code).double()
    return code * pick(s[name + "_scale"]).double()[..., e // case["group"]]


def _exact_read(case, s):
    page, at = s["slots"] // case["page"], s["slots"] % case["page"]
    # products of 4 and 24 bits are exact in 64
    return tuple(_exact_gather(case, s, n, page, at) for n in ("k", "v"))


def _exact_attention(case, s):
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEVICE)
    logs = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device=DEVICE)
    per, first = case["q_heads"] // case["kv_heads"], 0
    for b, (kv, q) in enumerate(zip(*_lengths(case))):
        if kv:
            j = torch.arange(kv, device=DEVICE)
            page, at = s["page_table"][b].long()[j // case["page"]], j % case["page"]
            hidden = None
            if case["causal"]:
                back = torch.arange(kv - q, kv, device=DEVICE)[:, None] - j
                hidden = (back < 0) | (back >= (case["window"] or kv + 1))
            for h in range(case["kv_heads"]):
                k = _exact_gather(case, s, "k", page, at, h)
                v = _exact_gather(case, s, "v", page, at, h)
                for r in range(h * per, (h + 1) * per):
                    x = s["q"][first:first + q, r].double() @ k.t() * s["scale"]
                    if hidden is not None:
                        x = x.masked_fill(hidden, -math.inf)
                    logs[first:first + q, r] = torch.logsumexp(x, -1)
                    out[first:first + q, r] = torch.nan_to_num(torch.softmax(x, -1)) @ v
        first += q
    return out, logs

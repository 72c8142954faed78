"""The operators of the feed-forward block in 8-bit floating point, as they are measured.

The products next to the int8 ones, with a scale for each block of 128, and what
makes their operands:

* ``norm``: the residual's addition and the root-mean-square norm in front of a
  linear layer, with its output in 8 bits: e4m3 in blocks of 128, or int8 per
  token or per group, which then go into the int8 product that takes them;
* ``product``: x [tokens, width] times weights [features, width], both e4m3,
  x with a scale for 128 consecutive values, the weights for 128 x 128;
* ``linear``: the same from fp16 activations, quantised on the way;
* ``gated``: act(x Wg^T) * (x Wu^T), the first half of a gated feed-forward
  block, its output fp16;
* ``block``: both halves, x [tokens, width] through ``features`` inner values
  and back to ``width``: the gated product with its output again e4m3 in blocks
  of 128, and the product that takes it.

Formats.  e4m3 codes with fp32 scales: s = fl32(amax / 448), code =
e4m3(fl32(x / s)) to nearest even, a block of zeros has s = 0.  Activations'
scales lie with the tokens side by side, [ceil(width / 128), tokens]; weights'
are [ceil(features / 128), ceil(width / 128)].  The int8 rule: s =
fl32(amax / 127), code = round_half_away(fl32(x / s)).
"""
from __future__ import annotations

import math

import torch

own = False

DEVICE = "cuda"
BLOCK = 128
EPS = 1e-6


# --------------------------------------------------------------------------- cases

def _norm(name, tokens, width, residual, form, group=0, features=0):
    return dict(name=name, op="norm", tokens=tokens, width=width, residual=residual, form=form, group=group,
                features=features)


def _product(name, op, tokens, features, width):
    return dict(name=name, op=op, tokens=tokens, features=features, width=width)


def _gated(name, op, tokens, features, width, activation):
    return dict(name=name, op=op, tokens=tokens, features=features, width=width, activation=activation)


def listed():
    return [
        # one generated token: the norm in front of its feed-forward block, latency alone counts
        _norm("norm 1 x 4096", 1, 4096, True, "f8"),
        # the 4516-token prompt of the W4A8 decoder layer
        _norm("norm 4516 x 4096", 4516, 4096, True, "f8"),
        # a step of 32 sequences: the norm into the int8 product that stands behind it
        _norm("norm 32 x 2560 to int8", 32, 2560, True, "int8", 0, 10240),
        # part of a prompt through a square layer (o), fp16 in and out
        _product("linear 517 x 4096 x 4096", "linear", 517, 4096, 4096),
        # one generated token through the down product: the weights are read once
        _product("product 1 x 4096 x 12288", "product", 1, 4096, 12288),
        # a step of 32 sequences
        _product("product 32 x 10240 x 2560", "product", 32, 10240, 2560),
        # the headline layer of the int8 products
        _product("product 4096 x 10240 x 2560", "product", 4096, 10240, 2560),
        # the prompt through the down product
        _product("product 4516 x 4096 x 12288", "product", 4516, 4096, 12288),
        # part of a prompt through gate and up, a share of odd size, the other activation
        _gated("gated 301 x 5121 x 2560", "gated", 301, 5121, 2560, "gelu_tanh"),
        # one generated token through the whole feed-forward block
        _gated("block 1 x 12288 x 4096", "block", 1, 12288, 4096, "silu"),
        # a step of 64 sequences, the wider feed-forward block
        _gated("block 64 x 14336 x 4096", "block", 64, 14336, 4096, "silu"),
        # the prompt through it
        _gated("block 4516 x 12288 x 4096", "block", 4516, 12288, 4096, "silu"),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(("norm", "norm", "linear", "product", "product", "gated", "block", "block"))
    tokens = _log(rng, 1, 8192)
    if op == "norm":
        form = rng.choice(("f8", "f8", "int8", "int8"))
        most = min(16384, 4516 * 4096 // tokens)
        if form == "f8":
            case = _norm("", tokens, 16 * _log(rng, 4, most // 16), rng.random() < 0.7, form)
        else:
            group = rng.choice((0, 0, 64, 128))
            width = 128 * _log(rng, 1, most // 128)
            case = _norm("", tokens, width, rng.random() < 0.7, form, group, 4 * _log(rng, 4, 1024))
    else:
        width = 16 * _log(rng, 4, 1024)
        sides = {"gated": 2, "block": 3}.get(op, 1)
        features = _log(rng, 16, min(16384, 3 * 4516 * 12288 * 4096 // (tokens * width * sides)))
        if sides > 1:
            # the block's inner values are the next product's operand: a multiple of 16 of them
            case = _gated("", op, tokens, features - features % 16 if op == "block" else features, width,
                          rng.choice(("silu", "silu", "gelu_tanh")))
        else:
            case = _product("", op, tokens, features, width)
    case.pop("name")
    return case


# --------------------------------------------------------------------------- what a case holds

def _blocks(n):
    return -(-n // BLOCK)


def work(case):
    m, k = case["tokens"], case["width"]
    if case["op"] == "norm":
        values = m * k
        bytes_ = 2 * values + 2 * k                                    # the rows and the gains in
        flops = 6 * values                                             # square and sum, gain, largest, quotient
        if case["residual"]:
            bytes_, flops = bytes_ + 4 * values, flops + values        # the residual in and out
        if case["form"] == "f8":
            bytes_ += values + 4 * m * _blocks(k)
        else:                                                          # the codes end in the product
            n = case["features"]
            groups = k // case["group"] if case["group"] else 1
            bytes_ += n * k + 4 * n * groups + 2 * m * n
            flops += 2 * m * n * k
        return {"bytes": bytes_, "flops": flops}
    n = case["features"]
    sides = {"gated": 2, "block": 3}.get(case["op"], 1)
    bytes_ = sides * (n * k + 4 * _blocks(n) * _blocks(k))
    bytes_ += 2 * m * k if case["op"] == "linear" else m * k + 4 * m * _blocks(k)
    bytes_ += 2 * m * (k if case["op"] == "block" else n)
    return {"bytes": bytes_, "flops": 2 * sides * m * n * k}


# --------------------------------------------------------------------------- inputs

def _generator(seed):
    return torch.Generator(device=DEVICE).manual_seed(int(seed))


def _rows(tokens, width, g):
    """Activations: a few channels and a few tokens are many times the others."""
    x = torch.randn(tokens, width, device=DEVICE, generator=g)
    x[:, 5::331] *= 20
    x[3::97] *= 8
    return x.half()


def _weights(features, width, g):
    return (torch.randn(features, width, device=DEVICE, generator=g) * 0.02).half()


def _in_blocks(x, rows, columns):
    """[R, C] as [R', rows, C', columns], zeros past the ends."""
    r, c = x.shape
    x = torch.nn.functional.pad(x, (0, -c % columns, 0, -r % rows))
    return x.reshape(-1, rows, x.shape[1] // columns, columns)


def _quotient(x, s):
    """fl32(x / s), zero where s is: the quotient in 64 bits, rounded once."""
    s = s.double()
    return torch.where(s > 0, x.double() / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(s)).float()


def _to_f8(x, rows):
    """fp32 [R, C] in blocks of rows x 128: (codes [R, C], scales [ceil(R / rows), ceil(C / 128)])."""
    b = _in_blocks(x, rows, BLOCK)
    s = (b.abs().amax((1, 3), keepdim=True).double() / 448).float()
    q = _quotient(b, s).flatten(2).flatten(0, 1)[:x.shape[0], :x.shape[1]]
    return q.to(torch.float8_e4m3fn), s[:, 0, :, 0]


def _to_int8(x, group):
    """fp32 [R, C] in groups along a row: (codes as fp32 [R, C], scales [R, groups])."""
    b = x.unflatten(1, (-1, group))
    s = (b.abs().amax(-1, keepdim=True).double() / 127).float()
    t = _quotient(b, s)
    whole = torch.trunc(t)
    q = whole + torch.sign(t) * ((t - whole).abs() >= 0.5)
    return q.clamp(-127, 127).flatten(1), s[..., 0]


def prepare(case, seed):
    g = _generator(seed)
    state = dict(case)
    m, k, op = case["tokens"], case["width"], case["op"]
    if op == "norm":
        state["x"] = _rows(m, k, g)
        state["gain"] = (1 + 0.2 * torch.randn(k, device=DEVICE, generator=g)).half()
        state["stream"] = _rows(m, k, g) * 3 if case["residual"] else None
        if case["form"] == "int8":
            q, s = _to_int8(_weights(case["features"], k, g).float(), case["group"] or k)
            state["w"], state["w_scale"] = q.to(torch.int8), (s if case["group"] else s[:, 0]).contiguous()
        return state
    n = case["features"]
    x = _rows(m, k, g)
    if op == "linear":
        state["x"] = x
    else:
        q, s = _to_f8(x.float(), 1)
        state["xq"], state["x_scale"] = q, s.t().contiguous()
    shapes = {"gate": (n, k), "up": (n, k), "down": (k, n)} if op == "block" else {"gate": (n, k), "up": (n, k)}
    for side, shape in shapes.items() if op in ("gated", "block") else (("w", (n, k)),):
        state[side], s = _to_f8(_weights(*shape, g).float(), BLOCK)
        state[side + "_scale"] = s.contiguous()
    if own:
        # what a program keeps next to its weights: the workspaces
        import w4a8_int8_gemm_amd as w
        if op == "product":
            state["workspace"] = w.f8_gemm_workspace(m, n, k)
        elif op != "linear":
            state["workspace"] = w.f8_gemm_gated_workspace(m, n, k, quantize=op == "block")
            if op == "block":
                state["workspace_down"] = w.f8_gemm_workspace(m, k, n)
        else:
            size = w.linear_workspace_size(w.Mode.F8, m, k)
            state["workspace"] = torch.empty(max(1, size), dtype=torch.uint8, device=DEVICE)
    return state


# --------------------------------------------------------------------------- one pass

def run(state):
    op = state["op"]
    if own:
        import w4a8_int8_gemm_amd as w
        if op == "norm":
            if state["form"] == "f8":
                return w.rmsnorm_quant(w.Mode.F8, state["x"], state["gain"], EPS, residual=state["stream"])
            mode = w.Mode.W8A8_PG if state["group"] else w.Mode.W8A8_PC
            q, s, *stream = w.rmsnorm_quant(mode, state["x"], state["gain"], EPS, residual=state["stream"],
                                            group_size=state["group"])
            if state["group"]:
                y = w.w8a8_gemm_pg(q, s, state["w"], state["w_scale"], state["group"])
            else:
                y = w.w8a8_gemm_pc(q, s, state["w"], state["w_scale"])
            return (y, *stream)
        if op == "linear":
            return w.linear(w.Mode.F8, state["x"], state["w"], state["w_scale"], workspace=state["workspace"])
        if op == "product":
            return w.f8_gemm(state["xq"], state["x_scale"], state["w"], state["w_scale"],
                             workspace=state["workspace"])
        out = w.f8_gemm_gated(state["xq"], state["x_scale"], state["gate"], state["gate_scale"], state["up"],
                              state["up_scale"], activation=state["activation"], quantize=op == "block",
                              workspace=state["workspace"])
        if op == "gated":
            return out
        return w.f8_gemm(*out, state["down"], state["down_scale"], workspace=state["workspace_down"])
    if op == "norm":
        return _plain_norm(state)
    if op == "linear":
        q, s = _to_f8(state["x"].float(), 1)
        return _plain_product(_plain_rows(q, s.t()), state, "w").half()
    x = _plain_rows(state["xq"], state["x_scale"])
    if op == "product":
        return _plain_product(x, state, "w").half()
    y = _plain_gated(x, state)
    if op == "gated":
        return y.half()
    q, s = _to_f8(y, 1)
    return _plain_product(_plain_rows(q, s.t()), state, "down").half()


def _plain_norm(state):
    h = state["x"].float()
    if state["residual"]:
        h = h + state["stream"].float()
    y = h / torch.sqrt((h * h).mean(-1, keepdim=True) + EPS) * state["gain"].float()
    if state["form"] == "f8":
        q, s = _to_f8(y, 1)
        out = (q, s.t().contiguous())
    else:
        group = state["group"] or state["width"]
        q, s = _to_int8(y, group)
        w = state["w"].float().unflatten(1, (-1, group)) * state["w_scale"].reshape(len(state["w"]), -1, 1)
        out = (torch.matmul((q.unflatten(1, (-1, group)) * s[..., None]).flatten(1), w.flatten(1).t()).half(),)
    return out + (h.half(),) if state["residual"] else out


def _plain_rows(codes, scale):
    """The values of activations' codes, their scales [blocks, tokens]."""
    return codes.float() * scale.t().repeat_interleave(BLOCK, 1)[:, :codes.shape[1]]


def _plain_product(x, state, side):
    w, s = state[side].float(), state[side + "_scale"]
    w = w * s.repeat_interleave(BLOCK, 0)[:w.shape[0]].repeat_interleave(BLOCK, 1)[:, :w.shape[1]]
    return torch.matmul(x, w.t())


def _plain_gated(x, state):
    a, b = _plain_product(x, state, "gate"), _plain_product(x, state, "up")
    if state["activation"] == "silu":
        a = a / (1 + torch.exp(-a))
    else:
        a = 0.5 * a * (1 + torch.tanh(math.sqrt(2 / math.pi) * (a + 0.044715 * a * a * a)))
    return a * b


# --------------------------------------------------------------------------- the same from the definitions, in 64 bits

def exact(case, seed):
    if case["op"] == "block":
        # the inner values are rounded to 8 bits on the way, and one next to a border between two codes may go
        # either way: whole steps of 2^-3 follow from differences in the last bits, so the output has no one
        # value; its two products are held to theirs by the other cases
        return None
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(case, s)
    if case["op"] == "linear":
        return _exact_values(s["x"].double())[0] @ _exact_weights(s, "w").t()
    k = case["width"]
    block = torch.arange(k, device=DEVICE) // BLOCK
    x = s["xq"].double() * s["x_scale"].double().index_select(0, block).t()
    if case["op"] == "product":
        return x @ _exact_weights(s, "w").t()
    g = x @ _exact_weights(s, "gate").t()
    if case["activation"] == "silu":
        g = g * torch.sigmoid(g)
    else:
        g = torch.nn.functional.gelu(g, approximate="tanh")
    return g * (x @ _exact_weights(s, "up").t())


def _exact_weights(s, side):
    """Every block of the weights by its own scale."""
    w = s[side].double()
    for i in range(0, w.shape[0], BLOCK):
        w[i:i + BLOCK] *= s[side + "_scale"][i // BLOCK].double().repeat(BLOCK, 1).t().flatten()[:w.shape[1]]
    return w


def _exact_parts(y):
    """What codes and scales of y [R, C] stand for before their rounding: (y / s, s), s [blocks, R]."""
    parts, scales = [], []
    for at in range(0, y.shape[1], BLOCK):
        p = y[:, at:at + BLOCK]
        s = torch.linalg.vector_norm(p, ord=math.inf, dim=1) / 448
        parts.append(torch.nan_to_num(p / s[:, None]))
        scales.append(s)
    return torch.cat(parts, 1), torch.stack(scales)


def _exact_values(x):
    """What fp16 activations stand for after the rule, whose roundings are part of the product's definition."""
    parts = []
    for at in range(0, x.shape[1], BLOCK):
        p = x[:, at:at + BLOCK]
        s = (torch.linalg.vector_norm(p, ord=math.inf, dim=1, keepdim=True) / 448).float().double()
        t = torch.nan_to_num(p / s).float().double()
        # e4m3: four significant bits down to 2^-6, steps of 2^-9 below
        step = torch.exp2(torch.clamp(torch.floor(torch.log2(torch.clamp(t.abs(), min=2.0 ** -20))), min=-6) - 3)
        parts.append(torch.round(t / step) * step * s)
    return (torch.cat(parts, 1),)


def _exact_norm(case, s):
    h = s["x"].double()
    if case["residual"]:
        h = h + s["stream"].double()
    k = case["width"]
    size = torch.linalg.vector_norm(h, dim=1, keepdim=True)
    y = h * torch.rsqrt(size * size / k + EPS) * s["gain"].double()
    if case["form"] == "f8":
        out = _exact_parts(y)
    else:
        # the codes' rounding is part of the definition; it is taken from 64-bit quotients
        group, parts = case["group"] or k, []
        for at in range(0, k, group):
            p = y[:, at:at + group]
            a = torch.linalg.vector_norm(p, ord=math.inf, dim=1, keepdim=True) / 127
            t = torch.nan_to_num(p / a)
            parts.append(torch.copysign(torch.floor(t.abs() + 0.5), t) * a)
        w = s["w"].double() * s["w_scale"].double().reshape(len(s["w"]), -1).repeat_interleave(group, 1)
        out = (torch.cat(parts, 1) @ w.t(),)
    return (*out, h) if case["residual"] else out

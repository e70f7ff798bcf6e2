"""What the operators between a decoder block's projections are measured on.

Each case is one pass through an operator: rotary positions of queries and keys, the norms before and after a block with
its gate and residual, the gated activation between a block's projections, and a mixture-of-experts layer over quantized
experts for a few tokens.  `run` computes it either in elementary torch operations (the plain form, `own` false) or
through the framework's entry points (`own` true).

Experts are held as the base weights are, all experts of a matrix one after the other ([experts * rows][columns]):
  q8_0: qs int8 [rows][columns], d binary16 [rows][columns / 32]; weight = d * q.
  q4_0: qs uint8 [rows][columns / 2], byte p of a row holds element 2p in its low and 2p + 1 in its high half; d as for
        q8_0; weight = d * (code - 8).
  q4_K: qs as q4_0; 16 bytes [rows][columns / 256][16] in the place of d: binary16 d and dmin, eight 6-bit scales sc and
        eight 6-bit minimums m as 48-bit little-endian fields; weight = d * sc * code - dmin * m, sc and m by 32 columns.
"""
import math

import torch

own = False

BF16, F32 = "bf16", "f32"
DTYPE = {BF16: torch.bfloat16, F32: torch.float32}
SIZE = {BF16: 2, F32: 4}
Q8_0, Q4_0, Q4_K = "q8_0", "q4_0", "q4_K"
# bytes of 256 weights
PACKED = {Q8_0: 256 + 16, Q4_0: 128 + 16, Q4_K: 128 + 16}


# ---------------------------------------------------------------- the cases

def listed():
    rope = dict(op="rope", heads=32, kv=8, dim=128, rot=128, layout="half", base=500000.0, scaling="none", factor=1.0,
                original=0, far=8192)
    norm = dict(op="norm", norm="rms", post="none", gate="none", alpha=1.0, beta=1.0, offset=0.0, bias=False)
    moe = dict(op="moe", score="softmax", renormalize=True, bias=False, given=False, scale=1.0, act="silu")
    return [
        # a decode step of eight sequences far into long contexts: projections' fp32 outputs, bf16 for the attention
        dict(rope, name="rope decode 8", tokens=8, dtype=F32, out=BF16, scaling="bands", factor=8.0, original=8192,
             far=120000),
        # prompts of a batch, in the type of the cache's attention
        dict(rope, name="rope prompts", tokens=8192, dtype=BF16, out=BF16, scaling="ramp", factor=4.0, original=32768,
             far=131072),
        # a part of the head in neighbouring pairs, fp32 throughout, an odd number of tokens and heads
        dict(rope, name="rope part pairs", tokens=5003, heads=9, kv=3, dim=96, rot=40, layout="pairs", dtype=F32,
             out=F32, base=10000.0, scaling="linear", factor=4.0),
        # one token between two blocks: the projection's fp32 output joins a bf16 residual
        dict(norm, name="norm decode 1", tokens=1, hidden=4096, x=BF16, y=F32, out=BF16),
        # prompts, norms on both sides of the block
        dict(norm, name="norm prompts", tokens=8192, hidden=4096, x=BF16, y=F32, out=BF16, post="rms", offset=1.0),
        # layer norms with gates of each sequence, odd width, residual scale
        dict(norm, name="norm gated odd", tokens=3001, hidden=1155, x=F32, y=F32, out=F32, norm="layer", post="layer",
             gate="rows", alpha=0.9, beta=1.25, bias=True),
        # one token of the 8B block's feed-forward part, and a prompt of it
        dict(op="glu", name="glu decode 1", tokens=1, ffn=14336, act="silu", dtype=F32, out=BF16),
        dict(op="glu", name="glu prompt", tokens=4096, ffn=14336, act="gelu_tanh", dtype=BF16, out=BF16),
        # one token, few large experts of the 8B block's shape
        dict(moe, name="moe decode 1 large", tokens=1, quant=Q8_0, experts=8, top=2, hidden=4096, ffn=14336, dtype=F32),
        # one token, many small experts
        dict(moe, name="moe decode 1 small", tokens=1, quant=Q4_0, experts=128, top=8, hidden=2048, ffn=768,
             dtype=BF16),
        # a ragged batch, sigmoid scores with a bias for the choice
        dict(moe, name="moe 19 tokens", tokens=19, quant=Q4_K, experts=64, top=6, hidden=2048, ffn=1280, dtype=BF16,
             score="sigmoid", bias=True, scale=2.5),
        # decode of 64 sequences: almost every expert is chosen by someone
        dict(moe, name="moe 64 tokens", tokens=64, quant=Q4_0, experts=128, top=8, hidden=2048, ffn=768, dtype=BF16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rope", "norm", "glu", "moe", "moe"))
    if op == "rope":
        dim = rng.choice((64, 80, 96, 128, 256))
        kv = rng.choice((1, 2, 3, 8))
        case = dict(op=op, tokens=_log(rng, 1, 8192), kv=kv, heads=kv * rng.choice((1, 3, 4)), dim=dim,
                    rot=rng.choice((dim, dim, dim // 2, 2 * rng.randint(8, dim // 2))), layout=rng.choice(("half", "pairs")),
                    base=rng.choice((10000.0, 500000.0, 1000000.0)), dtype=rng.choice((F32, BF16)),
                    out=rng.choice((F32, BF16)), far=_log(rng, 64, 1000000),
                    scaling=rng.choice(("none", "linear", "base", "bands", "ramp")), factor=rng.uniform(1.5, 16.0),
                    original=rng.choice((4096, 8192, 32768)))
        while case["tokens"] * (case["heads"] + kv) * dim > 8192 * 40 * 128:
            case["tokens"] //= 2
        return case
    if op == "norm":
        case = dict(op=op, tokens=_log(rng, 1, 8192), hidden=rng.choice((rng.randint(64, 8192), 8 * rng.randint(8, 1024))),
                    x=rng.choice((F32, BF16)), y=rng.choice((F32, BF16)), out=rng.choice((F32, BF16)),
                    norm=rng.choice(("rms", "layer")), post=rng.choice(("none", "rms", "layer")),
                    gate=rng.choice(("none", "channels", "rows")), alpha=rng.choice((1.0, rng.uniform(0.5, 1.5))),
                    beta=rng.choice((1.0, rng.uniform(0.2, 2.0))), offset=rng.choice((0.0, 1.0)),
                    bias=rng.choice((False, True)))
        while work(case)["bytes"] > 350e6:
            case["tokens"] //= 2
        return case
    if op == "glu":
        case = dict(op=op, tokens=_log(rng, 1, 4096), ffn=_log(rng, 64, 16384), act=rng.choice(("silu", "gelu", "gelu_tanh", "relu")),
                    dtype=rng.choice((F32, BF16)), out=rng.choice((F32, BF16)))
        while case["tokens"] * case["ffn"] * (2 * SIZE[case["dtype"]] + SIZE[case["out"]]) > 4096 * 14336 * 6:
            case["tokens"] //= 2
        return case
    quant = rng.choice((Q8_0, Q4_0, Q4_K))
    unit = 256 if quant == Q4_K else 32
    experts = rng.choice((4, 8, 16, 60, 128, 256))
    case = dict(op=op, tokens=_log(rng, 1, 64), quant=quant, experts=experts, top=rng.randint(1, min(8, experts)),
                hidden=unit * rng.randint(512 // unit, 4096 // unit), ffn=unit * max(1, round(_log(rng, 256, 8192) / unit)),
                dtype=rng.choice((F32, BF16)), score=rng.choice(("softmax", "sigmoid")),
                renormalize=rng.choice((False, True)), bias=rng.choice((False, True)),
                given=rng.random() < 0.2, scale=rng.choice((1.0, 2.5)), act=rng.choice(("silu", "gelu_tanh")))
    # bounds on what is held, and on what one pass costs
    while case["experts"] * case["hidden"] * case["ffn"] > 8 * 4096 * 14336:
        case["ffn"] = max(unit, case["ffn"] // 2 // unit * unit)
    while work(case)["bytes"] > 350e6 or work(case)["flops"] > 5e9:
        if case["tokens"] > 1:
            case["tokens"] //= 2
        else:
            case["top"] -= 1
    return case


def work(case):
    t = case["tokens"]
    if case["op"] == "rope":
        n = t * (case["heads"] + case["kv"]) * case["dim"]
        return {"bytes": n * (SIZE[case["dtype"]] + SIZE[case["out"]]) + 4 * t, "flops": 3 * n}
    if case["op"] == "norm":
        n = t * case["hidden"]
        gates = {"none": 0, "channels": 1, "rows": min(t, 8)}[case["gate"]] * case["hidden"] * 4
        return {"bytes": n * (2 * SIZE[case["x"]] + SIZE[case["y"]] + SIZE[case["out"]]) + gates + 4 * case["hidden"],
                "flops": 12 * n}
    if case["op"] == "glu":
        n = t * case["ffn"]
        return {"bytes": n * (2 * SIZE[case["dtype"]] + SIZE[case["out"]]), "flops": 10 * n}
    e, k, h, f = (case[n] for n in ("experts", "top", "hidden", "ffn"))
    some = e * (1 - (1 - k / e) ** t)                           # experts that someone chooses, evenly spread choices
    weights = 3 * h * f * PACKED[case["quant"]] / 256
    router = 0 if case["given"] else 4 * e * h
    return {"bytes": int(some * weights + router + 2 * t * h * SIZE[case["dtype"]]),
            "flops": 6 * t * k * h * f + (0 if case["given"] else 2 * t * e * h)}


# ---------------------------------------------------------------- inputs

def _random_experts(case, rows, columns, g):
    """One matrix of every expert, weights of about 1 / sqrt(columns) in size."""
    n = case["experts"] * rows
    size = 1 / math.sqrt(columns)
    dev = torch.device("cuda")
    spread = torch.rand((n, columns // (256 if case["quant"] == Q4_K else 32)), generator=g, device=dev) + 0.5
    if case["quant"] == Q8_0:
        qs = torch.randint(-127, 128, (n, columns), generator=g, device=dev, dtype=torch.int8)
        return qs, (spread * (size / 73)).half()
    qs = torch.randint(0, 256, (n, columns // 2), generator=g, device=dev, dtype=torch.uint8)
    if case["quant"] == Q4_0:
        return qs, (spread * (size / 4.6)).half()
    # sub-blocks' scales and minimums: 7.5 codes up from the minimum is zero on the average
    head = torch.randint(0, 256, (*spread.shape, 16), generator=g, device=dev, dtype=torch.uint8)
    d = (spread * (size / 160)).half()
    head[..., :4] = torch.stack((d, (d.float() * 7.5).half()), -1).view(torch.uint8)
    return qs, head


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(int(seed))
    dev = torch.device("cuda")

    def normal(*shape, dtype=F32):
        return torch.randn(shape, generator=g, device=dev).to(DTYPE[dtype])

    st = {"case": case}
    t = case["tokens"]
    if case["op"] == "rope":
        # queries and keys lie side by side, as one projection writes them
        st["qk"] = normal(t, case["heads"] + case["kv"], case["dim"], dtype=case["dtype"])
        st["q"], st["k"] = st["qk"][:, :case["heads"]], st["qk"][:, case["heads"]:]
        st["pos"] = torch.randint(0, case["far"], (t,), generator=g, device=dev, dtype=torch.int32)
    elif case["op"] == "norm":
        h = case["hidden"]
        # a few channels of a residual stream are far larger than the rest
        big = torch.where(torch.rand(h, generator=g, device=dev) < 0.01, 30.0, 1.0)
        st["x"] = (normal(t, h) * big + 0.2).to(DTYPE[case["x"]])
        st["y"] = (normal(t, h) * 0.5).to(DTYPE[case["y"]])
        st["weight"] = 1 - case["offset"] + 0.2 * normal(h)
        st["post_weight"] = 1 - case["offset"] + 0.2 * normal(h)
        st["bias"], st["post_bias"] = 0.1 * normal(h), 0.1 * normal(h)
        if case["gate"] == "channels":
            st["gate"] = normal(h)
        if case["gate"] == "rows":                              # one gate a sequence of the packed batch
            st["gate"] = normal(min(t, 8), h)
            st["gate_row"] = torch.randint(0, min(t, 8), (t,), generator=g, device=dev).sort().values.int()
    elif case["op"] == "glu":
        st["gate"], st["up"] = normal(t, case["ffn"], dtype=case["dtype"]), normal(t, case["ffn"], dtype=case["dtype"])
    else:
        e, k, h, f = (case[n] for n in ("experts", "top", "hidden", "ffn"))
        st["gate"], st["up"] = _random_experts(case, f, h, g), _random_experts(case, f, h, g)
        st["down"] = _random_experts(case, h, f, g)
        st["x"] = normal(t, h, dtype=case["dtype"])
        st["router"] = normal(e, h) * (1.5 / math.sqrt(h))
        st["bias"] = 0.1 * normal(e) if case["bias"] else None
        if case["given"]:                                       # a choice made elsewhere; some places are left empty
            choice = torch.rand((t, e), generator=g, device=dev).argsort(-1)[:, :k].int()
            choice[torch.rand((t, k), generator=g, device=dev) < 0.15] = -1
            st["choice"], st["weight"] = choice, torch.rand((t, k), generator=g, device=dev)
    return st


# ---------------------------------------------------------------- the plain form

def _frequencies(case, device):
    """Radians a position of every pair, float64 [rot / 2], and the factor of both cosine and sine."""
    rot, base, s, original = case["rot"], case["base"], case["factor"], case["original"]
    i = torch.arange(rot // 2, dtype=torch.float64, device=device)
    if case["scaling"] == "base" and rot > 2:
        base = base * s ** (rot / (rot - 2))
    f = base ** (-2 * i / rot)
    if case["scaling"] == "linear":
        return f / s, 1.0
    if case["scaling"] == "bands":                              # 1 and 4 turns within the original length
        turns = original * f / (2 * math.pi)
        keep = ((turns - 1) / 3).clamp(0, 1)
        return f * keep + f / s * (1 - keep), 1.0
    if case["scaling"] == "ramp":                               # 32 turns and 1 turn, by the pair's number
        at = [rot * math.log(original / (2 * math.pi * turns)) / (2 * math.log(base)) for turns in (32, 1)]
        lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
        far = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        return f * (1 - far) + f / s * far, 0.1 * math.log(s) + 1
    return f, 1.0


def _plain_rope(st):
    case = st["case"]
    rot = case["rot"]
    f, size = _frequencies(case, st["pos"].device)
    angle = st["pos"].double()[:, None] * f
    cos, sin = (angle.cos() * size).float()[:, None], (angle.sin() * size).float()[:, None]
    out = {}
    for name in ("q", "k"):
        x = st[name].float()
        y = x.clone()
        a, b = (x[..., :rot // 2], x[..., rot // 2:rot]) if case["layout"] == "half" else (x[..., :rot:2], x[..., 1:rot:2])
        u, v = a * cos - b * sin, a * sin + b * cos
        y[..., :rot] = torch.cat((u, v), -1) if case["layout"] == "half" else torch.stack((u, v), -1).flatten(-2)
        out[name] = y.to(DTYPE[case["out"]])
    return out


def _normed(x, kind, weight, bias, offset):
    if kind == "none":
        return x
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * (weight + offset)
    return x if bias is None else x + bias


def _plain_norm(st):
    case = st["case"]
    bias, post_bias = (st["bias"], st["post_bias"]) if case["bias"] else (None, None)
    z = _normed(st["y"].float(), case["post"], st["post_weight"], post_bias, case["offset"])
    if case["gate"] == "channels":
        z = z * st["gate"]
    if case["gate"] == "rows":
        z = z * st["gate"][st["gate_row"].long()]
    x = case["alpha"] * st["x"].float() + case["beta"] * z
    h = _normed(x, case["norm"], st["weight"], bias, case["offset"])
    return {"x": x.to(DTYPE[case["x"]]), "h": h.to(DTYPE[case["out"]])}


def _activated(x, act):
    if act == "silu":
        return x / (1 + torch.exp(-x))
    if act == "gelu":
        return x * 0.5 * (1 + torch.erf(x * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return x * 0.5 * (1 + torch.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x * x * x)))
    return x.clamp(min=0)


def _plain_glu(st):
    case = st["case"]
    return {"out": (_activated(st["gate"].float(), case["act"]) * st["up"].float()).to(DTYPE[case["out"]])}


def _sixes(head):
    """head uint8 [..., 16] -> the eight scales and the eight minimums, float32 [..., 8] each."""
    out = []
    for at in (4, 10):
        b = head[..., at:at + 6].int().unflatten(-1, (2, 3))    # four fields in three bytes
        w = b[..., 0] | (b[..., 1] << 8) | (b[..., 2] << 16)
        out.append(torch.stack((w, w >> 6, w >> 12, w >> 18), -1).bitwise_and(63).flatten(-2).float())
    return out


def _dequantized(case, planes, rows, some):
    """float32 [experts][rows][columns] of the experts `some` (None: all)."""
    qs, d = (p.unflatten(0, (case["experts"], rows)) for p in planes)
    if some is not None:
        qs, d = qs[some], d[some]
    if case["quant"] == Q8_0:
        return (qs.float().unflatten(-1, (-1, 32)) * d.float().unsqueeze(-1)).flatten(-2)
    code = torch.stack((qs & 15, qs >> 4), -1).flatten(-2).float().unflatten(-1, (-1, 32))
    if case["quant"] == Q4_0:
        return ((code - 8) * d.float().unsqueeze(-1)).flatten(-2)
    both = d[..., :4].contiguous().view(torch.float16).float()
    scale, least = _sixes(d)
    scale, least = (scale * both[..., :1]).flatten(-2), (least * both[..., 1:]).flatten(-2)
    return (code * scale.unsqueeze(-1) - least.unsqueeze(-1)).flatten(-2)


def _routed(st):
    """choice int64 [tokens][top], weight float32: the router's, or the caller's."""
    case = st["case"]
    if case["given"]:
        return st["choice"].long(), st["weight"] * (st["choice"] >= 0)
    z = st["x"].double() @ st["router"].double().T              # 64 bits: choices may be close
    score = torch.sigmoid(z) if case["score"] == "sigmoid" else torch.softmax(z, -1)
    order = score if st["bias"] is None else score + st["bias"]
    choice = torch.sort(order, dim=-1, descending=True, stable=True).indices[:, :case["top"]]
    weight = score.gather(-1, choice)
    if case["renormalize"]:
        weight = weight / weight.sum(-1, keepdim=True)
    return choice, (weight * case["scale"]).float()


def _plain_moe(st):
    case = st["case"]
    e, k, h, f, t = (case[n] for n in ("experts", "top", "hidden", "ffn", "tokens"))
    choice, weight = _routed(st)
    x = st["x"].float()
    if t * k <= e:                                              # the chosen experts, once for each choice
        some = choice.clamp(min=0).flatten()
        x = x.repeat_interleave(k, 0).unsqueeze(1)
        mixed = weight.flatten()[:, None, None]
    else:                                                       # every expert on every token
        some = None
        mixed = torch.zeros((t, e), device=x.device).scatter_add_(1, choice.clamp(min=0), weight).T.unsqueeze(-1)
    gate = x @ _dequantized(case, st["gate"], f, some).transpose(1, 2)
    up = x @ _dequantized(case, st["up"], f, some).transpose(1, 2)
    y = ((_activated(gate, case["act"]) * up) @ _dequantized(case, st["down"], h, some).transpose(1, 2)) * mixed
    y = y.unflatten(0, (t, k)).sum((1, 2)) if some is not None else y.sum(0)
    return {"out": y.to(DTYPE[case["dtype"]])}


PLAIN = {"rope": _plain_rope, "norm": _plain_norm, "glu": _plain_glu, "moe": _plain_moe}


# ---------------------------------------------------------------- one pass

def _made(st):
    """What a program makes once and keeps: the operator with its weights and constants."""
    import quantized_base_lora_gb300 as q
    from quantized_base_lora_gb300 import block
    case = st["case"]
    if case["op"] == "rope":
        return block.Rope(case["dim"], rot_dim=case["rot"], layout=case["layout"], base=case["base"],
                          scaling=case["scaling"], factor=case["factor"], original=case["original"])
    if case["op"] == "norm":
        bias, post_bias = (st["bias"], st["post_bias"]) if case["bias"] else (None, None)
        post = None if case["post"] == "none" else block.Norm(case["post"], st["post_weight"], post_bias, eps=1e-6,
                                                              offset=case["offset"])
        return block.BlockNorm(case["hidden"], block.Norm(case["norm"], st["weight"], bias, eps=1e-6,
                                                          offset=case["offset"]),
                               post=post, alpha=case["alpha"], beta=case["beta"])
    if case["op"] == "glu":
        return block.glu
    return block.Moe({Q8_0: q.OVL_Q8_0, Q4_0: q.OVL_Q4_0, Q4_K: q.OVL_Q4_K}[case["quant"]], case["experts"],
                     case["hidden"], case["ffn"], st["gate"], st["up"], st["down"], top_k=case["top"],
                     router=None if case["given"] else st["router"], bias=st["bias"], score=case["score"],
                     renormalize=case["renormalize"], scale=case["scale"], act=case["act"], max_tokens=64)


def run(st):
    case = st["case"]
    if not own:
        return PLAIN[case["op"]](st)
    made = st.get("made")
    if made is None:
        made = st["made"] = _made(st)
    if case["op"] == "rope":
        q, k = made(st["pos"], st["q"], st["k"], dtype=DTYPE[case["out"]])
        return {"q": q, "k": k}
    if case["op"] == "norm":
        x, h = made(st["x"], st["y"], gate=st.get("gate"), gate_row=st.get("gate_row"), dtype=DTYPE[case["out"]])
        return {"x": x, "h": h}
    if case["op"] == "glu":
        return {"out": made(st["gate"], st["up"], act=case["act"], dtype=DTYPE[case["out"]])}
    return {"out": made(st["x"], choice=st.get("choice"), weight=st.get("weight"))}


# ---------------------------------------------------------------- in 64 bits

def _exact_rope(st):
    case = st["case"]
    half = case["rot"] // 2
    base, s, length = case["base"], case["factor"], case["original"]
    turn, size = [], 1.0
    for i in range(half):                                       # pair by pair, on the host
        b = base * s ** (case["rot"] / (case["rot"] - 2)) if case["scaling"] == "base" and half > 1 else base
        w = math.pow(b, -i / half)
        if case["scaling"] == "linear":
            w /= s
        elif case["scaling"] == "bands":
            n = w * length / math.tau
            w = w if n >= 4 else w / s if n <= 1 else w * ((n - 1) / 3) + w / s * ((4 - n) / 3)
        elif case["scaling"] == "ramp":
            size = 1 + math.log(s) / 10
            first = max(0, math.floor(half * math.log(length / (32 * math.tau)) / math.log(base)))
            last = min(case["rot"] - 1, math.ceil(half * math.log(length / math.tau) / math.log(base)))
            far = min(1.0, max(0.0, (i - first) / max(0.001, last - first)))
            w = w * (1 - far) + w / s * far
        turn.append(w)
    phase = torch.exp(1j * st["pos"].double()[:, None, None] * torch.tensor(turn, dtype=torch.float64, device="cuda")) * size
    out = {}
    for name in ("q", "k"):
        y = st[name].double().clone()
        first = slice(0, half) if case["layout"] == "half" else slice(0, 2 * half, 2)
        second = slice(half, 2 * half) if case["layout"] == "half" else slice(1, 2 * half, 2)
        z = torch.complex(y[..., first], y[..., second]) * phase
        y[..., first], y[..., second] = z.real, z.imag
        out[name] = y
    return out


def _exact_norm(st):
    case = st["case"]

    def of(v, kind, w, b):
        if kind == "none":
            return v
        mid = v.mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(v[:, :1])
        var = (v - mid).pow(2).mean(1, keepdim=True)
        r = (v - mid) / torch.sqrt(var + 1e-6) * (w.double() + case["offset"])
        return r + b.double() if case["bias"] else r

    z = of(st["y"].double(), case["post"], st["post_weight"], st["post_bias"])
    if case["gate"] != "none":
        rows = st["gate"].double().reshape(-1, case["hidden"])
        z = rows.expand(len(z), -1) * z if case["gate"] == "channels" else rows.index_select(0, st["gate_row"].long()) * z
    x = st["x"].double() * case["alpha"] + z * case["beta"]
    return {"x": x, "h": of(x, case["norm"], st["weight"], st["bias"])}


def _exact_act(v, act):
    if act == "silu":
        return v * torch.special.expit(v)
    if act == "gelu":
        return v * torch.special.ndtr(v)
    if act == "gelu_tanh":                                      # (1 + tanh u) / 2 = 1 / (1 + exp(-2 u))
        return v * torch.special.expit(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))
    return torch.where(v > 0, v, torch.zeros_like(v))


def _exact_rows(case, planes, first, n):
    """float64 [n][columns] of the rows from `first`, one 32-weight block's formula at a time."""
    qs, d = planes[0][first:first + n], planes[1][first:first + n]
    if case["quant"] == Q8_0:
        return qs.double() * d.double().repeat_interleave(32, 1)
    w = torch.empty((n, 2 * qs.shape[1]), dtype=torch.float64, device=qs.device)
    w[:, 0::2], w[:, 1::2] = (qs % 16).double(), (qs // 16).double()
    if case["quant"] == Q4_0:
        return (w - 8) * d.double().repeat_interleave(32, 1)
    two = d[:, :, :4].contiguous().view(torch.float16).double()
    fields = [sum(d[:, :, at + i].long() << (8 * i) for i in range(6)) for at in (4, 10)]
    for j in range(8):
        sc, m = ((v >> (6 * j)) % 64 for v in fields)
        a, b = (two[:, :, 0] * sc).unsqueeze(-1), (two[:, :, 1] * m).unsqueeze(-1)
        part = w.view(n, -1, 8, 32)[:, :, j]
        part.mul_(a).sub_(b)
    return w


def _exact_moe(st):
    case = st["case"]
    e, k, h, f, t = (case[n] for n in ("experts", "top", "hidden", "ffn", "tokens"))
    x = st["x"].double()
    if case["given"]:
        pairs = [(i, c, w) for i, (cs, ws) in enumerate(zip(st["choice"].tolist(), st["weight"].tolist()))
                 for c, w in zip(cs, ws) if c >= 0]
    else:
        z = (x @ st["router"].double().T).cpu()
        pairs = []
        for i in range(t):
            p = torch.special.expit(z[i]) if case["score"] == "sigmoid" else torch.exp(z[i] - torch.logsumexp(z[i], 0))
            by = p + st["bias"].double().cpu() if case["bias"] else p
            top = sorted(range(e), key=lambda j: (-by[j].item(), j))[:k]
            total = sum(p[j].item() for j in top) if case["renormalize"] else 1.0
            pairs += [(i, j, p[j].item() / total * case["scale"]) for j in top]
    y = torch.zeros((t, h), dtype=torch.float64, device=x.device)
    for j in sorted({c for _, c, _ in pairs}):
        rows = [(i, w) for i, c, w in pairs if c == j]
        at = torch.tensor([i for i, _ in rows], device=x.device)
        w = torch.tensor([w for _, w in rows], dtype=torch.float64, device=x.device)
        u = _exact_act(x[at] @ _exact_rows(case, st["gate"], j * f, f).T, case["act"])
        u = u * (x[at] @ _exact_rows(case, st["up"], j * f, f).T)
        y.index_add_(0, at, (u @ _exact_rows(case, st["down"], j * h, h).T) * w[:, None])
    return {"out": y}


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(st)
    if case["op"] == "norm":
        return _exact_norm(st)
    if case["op"] == "glu":
        return {"out": _exact_act(st["gate"].double(), case["act"]) * st["up"].double()}
    return _exact_moe(st)

"""What the operators between a block's projections compute, in 64 bits, and how far 32-bit results may be from it."""
import math

import numpy as np
import torch

import oracle as O

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}       # half a step of an output, relative to the value


def frequencies(rot, base=10000.0, scaling=None, factor=1.0, original=0, low=None, high=None):
    """Radians a position of every pair, by the definition; and the magnitude."""
    if scaling == "base" and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    w = [base ** (-2 * i / rot) for i in range(rot // 2)]
    low, high = low or 1.0, high or {"bands": 4.0, "ramp": 32.0}.get(scaling, 4.0)
    if scaling == "linear":
        w = [v / factor for v in w]
    if scaling == "bands":
        out = []
        for v in w:
            n = original * v / math.tau
            s = min(1.0, max(0.0, (n - low) / (high - low)))
            out.append(s * v + (1 - s) * v / factor)
        w = out
    if scaling == "ramp":
        def at(n):
            return rot * math.log(original / (n * math.tau)) / (2 * math.log(base))
        a, b = max(0, math.floor(at(high))), min(rot - 1, math.ceil(at(low)))
        r = [min(1.0, max(0.0, (i - a) / max(b - a, 0.001))) for i in range(rot // 2)]
        return [v * (1 - x) + v / factor * x for v, x in zip(w, r)], 0.1 * math.log(factor) + 1
    return w, 1.0


def rope(x, pos, w, size, layout):
    """x [tokens][heads][dim] float64, and |a| + |b| of each pair (0 where channels are passed through)."""
    rot = 2 * len(w)
    ang = pos.double()[:, None, None] * torch.tensor(w, dtype=torch.float64, device=x.device)
    cos, sin = ang.cos() * size, ang.sin() * size
    y, mag = x.clone(), torch.zeros_like(x)
    i, j = (slice(0, rot // 2), slice(rot // 2, rot)) if layout == "half" else (slice(0, rot, 2), slice(1, rot, 2))
    a, b = x[..., i], x[..., j]
    y[..., i], y[..., j] = a * cos - b * sin, a * sin + b * cos
    mag[..., i] = mag[..., j] = (a.abs() + b.abs()) * size
    return y, mag


def rope_allowed(y, mag, dtype):
    """Sine and cosine: the angle, up to pi / 4, is rounded twice (2^-24 each) and cut to 2^-32 of a turn: 1.0e-7; the
    series end within 2e-9 and their last three steps round, 2^-24 each: 1.8e-7, with the factor's rounding 3.5e-7 in
    all, below 2^-21.  Two products and a sum: 2^-24 of each, so 2^-20.5 of |a| + |b|; the output's half step."""
    return mag * 2.0 ** -20.5 + y.abs() * HALF[dtype] * 1.001


def normed(v, kind, w, b, eps, offset):
    """(norm, how far the fp32 one may be): sums of n terms in a tree are off by 2^-19 of their terms' size at the
    widths here (32 rounded additions in a row at most), which goes into the mean, and by halves into the root."""
    if kind is None:
        return v, torch.zeros_like(v)
    mean = v.mean(-1, keepdim=True) if kind == "layer" else torch.zeros_like(v[..., :1])
    c = v - mean
    r = 1 / torch.sqrt(c.square().mean(-1, keepdim=True) + eps)
    g = torch.ones_like(v) if w is None else (w.double() + offset).expand_as(v)
    out = c * r * g
    off = 2.0 ** -19 * (r * g.abs() * (v.abs().mean(-1, keepdim=True) * (kind == "layer") + c.abs()) + out.abs())
    return (out if b is None else out + b.double()), off + (0 if b is None else 2.0 ** -23 * (out.abs() + b.double().abs()))


def activated(v, act):
    if act == "silu":
        return v * torch.special.expit(v)
    if act == "gelu":
        return v * torch.special.ndtr(v)
    if act == "gelu_tanh":
        return v * torch.special.expit(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))
    return v.clamp(min=0)


# |act(a) - act(b)| <= SLOPE |a - b|
SLOPE = 1.13


def experts(rng, quant, n, rows, cols):
    """Random experts of about 1 / sqrt(cols): planes (qs, d) as numpy arrays, weights float64 [n][rows][cols]."""
    size = 1 / math.sqrt(cols)
    total = n * rows
    if quant == O.Q8_0:
        qs = rng.integers(-127, 128, (total, cols), dtype=np.int8)
        d = (rng.uniform(0.5, 1.5, (total, cols // 32)) * size / 73).astype(np.float16)
        w = O.dequantize(quant, qs, d.view(np.uint16))
    elif quant == O.Q4_0:
        qs = rng.integers(0, 256, (total, cols // 2), dtype=np.uint8)
        d = (rng.uniform(0.5, 1.5, (total, cols // 32)) * size / 4.6).astype(np.float16)
        w = O.dequantize(quant, qs, d.view(np.uint16))
    else:
        qs = rng.integers(0, 256, (total, cols // 2), dtype=np.uint8)
        d = rng.integers(0, 256, (total, cols // 256, 16), dtype=np.uint8)
        scale = (rng.uniform(0.5, 1.5, (total, cols // 256)) * size / 160).astype(np.float16)
        d[..., 0:2] = scale[..., None].view(np.uint8).reshape(*scale.shape, 2)
        d[..., 2:4] = (scale * np.float16(7.5)).astype(np.float16)[..., None].view(np.uint8).reshape(*scale.shape, 2)
        w = O.dequantize(quant, qs, d)
    return (qs, d), torch.from_numpy(np.ascontiguousarray(w, np.float64)).reshape(n, rows, cols)


def route(x, router, bias, score, top, renormalize, scale):
    """choice [tokens][top], weight float64, and the least distance between an order that was taken and one that was not."""
    z = x.double() @ router.double().T
    p = torch.sigmoid(z) if score == "sigmoid" else torch.softmax(z, -1)
    by = p + bias.double() if bias is not None else z
    order = torch.sort(by, dim=-1, descending=True, stable=True)
    choice, w = order.indices[:, :top], p.gather(-1, order.indices[:, :top])
    gap = (order.values[:, top - 1] - order.values[:, top]).min().item() if by.shape[1] > top else math.inf
    if renormalize:
        w = w / w.sum(-1, keepdim=True)
    return choice.int(), w * scale, gap


def moe(x, gate, up, down, choice, weight, act, f32):
    """(y, how far the library's may be), float64, by tokens; weights float64 [experts][rows][cols] on the CPU.

    A product of the library is a sum of blocks in fp32: an MMA cuts off its sums at 2^-23 of its largest product,
    counted, for codes below 128, as if the code were 128, which is 16 times the 4-bit codes' largest: 2^-19 for one
    of the at most 18 in a row of a block, so 2^-15 of the sum of |w x| covers them with the other roundings.
    Activations go in as two bf16 parts, 2^-16 (fp32 calls: three, 2^-23)."""
    tau, part = 2.0 ** -15, 2.0 ** -23 if f32 else 2.0 ** -16
    y, off = torch.zeros_like(x), torch.zeros_like(x)
    for t in range(x.shape[0]):
        for e, w in zip(choice[t].tolist(), weight[t].tolist()):
            if not 0 <= e < gate.shape[0]:
                continue
            g, u = gate[e] @ x[t], up[e] @ x[t]
            dg, du = tau * (gate[e].abs() @ x[t].abs()), tau * (up[e].abs() @ x[t].abs())
            a = activated(g, act)
            h = a * u
            dh = SLOPE * dg * (u.abs() + du) + (a.abs() + SLOPE * dg) * du + h.abs() * (part + 2.0 ** -18)
            d = down[e]
            y[t] += w * (d @ h)
            off[t] += abs(w) * (d.abs() @ (dh + tau * h.abs()))
    return y, off

"""What the operators of the 4-bit key/value cache are measured on.

Each case is one pass through an operator: writing new tokens into the cache, attention over it, sequences that fork
and sequences that are compacted.  `run` computes it either in elementary torch operations (the plain form, `own`
false) or through the framework's entry points (`own` true); both work on the same packed cache.

The packed cache.  `codes` is uint8 [pages][layers][2][kv heads][page tokens * D / 2], `scales` binary16
[pages][layers][2][kv heads][page tokens][D / 32]; index 0 of the third axis holds the keys, 1 the values.  32
consecutive channels of a token share a scale d = max|x| / 8, and channel c is worth d * (code - 8).
  keys:   each token's row is D / 32 blocks of four 4-byte words; word w of block b lies at word w * (D / 32) + b of the
          row and holds channels 32 b + 8 w .. + 7, the first in the lowest 4 bits.
  values: each group of 8 tokens is [8][8 tokens][D / 16 bytes]; unit (g, token) holds channels g, g + 8, g + 16, ...,
          the first in the lowest 4 bits.
`table` int32 [sequences][columns] names the page of every run of page tokens, -1 where there is none; `length` int32
counts a sequence's tokens, `refs` int32 the rows that hold a page.
"""
import math

import numpy as np
import torch

own = False

BF16, F32 = "bf16", "f32"
DTYPE = {BF16: torch.bfloat16, F32: torch.float32}


# ---------------------------------------------------------------- the cases

def listed():
    block = dict(heads=32, kv=8, dim=128, page=64, layers=1)    # the attention of the 4096-wide decoder block
    return [
        # a decode step of a small server: one token for each of 8 sequences, the smallest call there is
        dict(block, name="append 8x1", op="append", seqs=8, new=1, low=100, high=2000, dtype=BF16),
        # a prompt batch being taken in: 16 prompts of ragged lengths
        dict(block, name="append prompts", op="append", seqs=16, new=1900, low=1900, high=4000, dtype=F32),
        # one user, a short conversation: latency alone
        dict(block, name="decode 1x1000", op="attend", seqs=1, new=1, low=1000, high=1000, dtype=F32, window=0, sinks=0),
        # an ordinary decode batch with ragged contexts
        dict(block, name="decode 32 ragged", op="attend", seqs=32, new=1, low=500, high=8000, dtype=BF16, window=0,
             sinks=0),
        # documents in context: the cache is what is read
        dict(block, name="decode 16 long", op="attend", seqs=16, new=1, low=60001, high=131072, dtype=BF16, window=0,
             sinks=0),
        # endless streams: a window and the first few tokens, the rest of the context unread
        dict(block, name="window decode 64", op="attend", seqs=64, new=1, low=1000, high=32768, dtype=BF16, window=2048,
             sinks=4),
        # a chunk of two prompts over what is already cached
        dict(block, name="prompt chunk 2x2048", op="attend", seqs=2, new=2048, low=6000, high=8192, dtype=BF16, window=0,
             sinks=0),
        # the same with a window, smaller heads and more queries to a key
        dict(name="window chunk 4x777", op="attend", heads=24, kv=3, dim=64, page=32, layers=1, seqs=4, new=777, low=777,
             high=6000, dtype=BF16, window=1024, sinks=4),
        # one sequence splits in two, one layer
        dict(block, name="fork 1", op="fork", seqs=1, low=1000, high=1000),
        # parallel samples of 24 prompts, all 32 layers of a model in one page
        dict(name="fork 24, 32 layers", op="fork", heads=32, kv=8, dim=128, page=64, layers=32, seqs=24, low=300,
             high=1000),
        # a context of 500 tokens loses half of them
        dict(block, name="compact 1", op="compact", seqs=1, low=500, high=500, keep=0.5),
        # eviction in a batch: a sequence keeps its first tokens, scattered ones and the latest
        dict(name="compact 16, 8 layers", op="compact", heads=32, kv=8, dim=128, page=64, layers=8, seqs=16, low=900,
             high=4000, keep=0.5),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    kv = rng.choice([1, 2, 3, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 7, 8])
    c = dict(heads=kv * group, kv=kv, dim=rng.choice([64, 128, 128, 256]), page=rng.choice([16, 32, 64, 128]))
    op = rng.choice(["append", "attend", "attend", "attend", "window", "window", "fork", "compact"])
    if op in ("attend", "window"):
        c.update(op="attend", layers=rng.choice([1, 1, 2]), dtype=rng.choice([BF16, BF16, F32]), window=0, sinks=0)
        c["new"] = rng.choice([1, 1, 1, _log(rng, 2, 9), _log(rng, 10, 1500)])
        high = _log(rng, max(16, c["new"]), 60000)
        # the plain form holds the cache in 32 bits and every score: both within some GB
        most = min(2.0e9 / (high * kv * c["dim"]), 1.5e9 / (high * c["new"] * c["heads"]))
        c["seqs"] = _log(rng, 1, max(1, min(64, int(most))))
        if most < 1:
            high = max(c["new"], int(high * most))
        c["low"], c["high"] = max(c["new"], _log(rng, max(1, high // 16), high)), high
        if op == "window":
            c["window"], c["sinks"] = _log(rng, 8, 4096), rng.choice([0, 1, 4, 5, 64])
        return c
    c["layers"] = rng.choice([1, 2, 4, 8])
    c["seqs"] = _log(rng, 1, 32)
    high = max(1, min(8000, int(2.0e8 / (c["seqs"] * c["layers"] * kv * c["dim"]))))
    if op == "append":
        c.update(op="append", layers=1, dtype=rng.choice([BF16, F32]), new=_log(rng, 1, high))
        c["low"], c["high"] = c["new"], max(c["new"], high)
    else:
        c["low"], c["high"] = _log(rng, 1, high), high
        c["op"] = op
        if op == "compact":
            c["keep"] = rng.choice([0.1, 0.5, 0.9])
    return c


def _lengths(case):
    """Tokens of each sequence and how many of them are new: plain numbers of the case alone."""
    r = np.random.RandomState(case["seqs"] * 7 + case["high"] % 1000)
    u = np.exp(r.uniform(math.log(case["low"]), math.log(case["high"]), case["seqs"])).round().astype(np.int64)
    length = np.clip(u, case["low"], case["high"])
    new = np.zeros_like(length)
    if case.get("new"):
        new += case["new"]
        if case["new"] > 1:                                     # ragged: some sequences bring fewer
            new[1::2] -= r.randint(0, case["new"] // 2 + 1, len(new[1::2]))
    return length, new


def _kept(case, length):
    """How many tokens of each sequence stay."""
    return [max(1, int(n * case["keep"])) for n in length]


def work(case):
    length, new = _lengths(case)
    heads, kv, dim = case["heads"], case["kv"], case["dim"]
    held = kv * (dim + dim // 8)                                # bytes of one token of one layer, keys and values
    if case["op"] == "append":
        size = 2 if case["dtype"] == BF16 else 4
        n = int(new.sum())
        # the input, the packed tokens, and the values they stand for
        return {"bytes": n * (2 * kv * dim * size + held + 2 * kv * dim * 4), "flops": n * 2 * kv * dim * 6}
    if case["op"] == "attend":
        size = 2 if case["dtype"] == BF16 else 4
        read = pairs = 0
        for n, t in zip(length.tolist(), new.tolist()):
            pos = np.arange(n - t, n, dtype=np.int64)
            seen = pos + 1
            if case["window"]:
                first = np.maximum(0, pos + 1 - case["window"])
                seen = seen - first + np.minimum(first, case["sinks"])
                lead = int(first[0])
                read += n - lead + min(lead, case["sinks"])
            else:
                read += n
            pairs += int(seen.sum())
        return {"bytes": read * held + 2 * int(new.sum()) * heads * dim * size, "flops": 4 * pairs * heads * dim}
    page = case["page"]
    if case["op"] == "fork":
        n = int((length % page != 0).sum()) * page              # whole pages are shared, the open one is copied
    else:
        n = sum(_kept(case, length.tolist()))
    return {"bytes": 2 * n * held * case["layers"], "flops": 0}


# ---------------------------------------------------------------- inputs

def _quantized(x):
    """x float32 [..., D] -> codes uint8 [..., D], scales binary16 [..., D / 32]."""
    b = torch.nan_to_num(x, nan=0.0, posinf=3.3e38, neginf=-3.3e38).unflatten(-1, (-1, 32))
    d = (b.abs().amax(-1) / 8).clamp(max=65504.0).half()
    s = d.float().unsqueeze(-1)
    q = torch.where(s > 0, b / s, torch.zeros_like(b))
    code = torch.trunc(q + torch.copysign(torch.full_like(q, 0.5), q)).clamp(-8, 7) + 8
    return code.to(torch.uint8).flatten(-2), d


def _packed_keys(code):
    """codes [..., P, D] -> bytes [..., P * D / 2]"""
    w = code.unflatten(-1, (-1, 4, 4, 2))                       # block, word, byte, nibble
    w = (w[..., 0] | (w[..., 1] << 4)).transpose(-3, -2)        # word, block, byte
    return w.flatten(-4)


def _packed_values(code):
    w = code.unflatten(-1, (-1, 2, 8)).unflatten(-4, (-1, 8))   # group, token, byte, nibble, c % 8
    w = w[..., 0, :] | (w[..., 1, :] << 4)                      # group, token, byte, c % 8
    return w.permute(*range(w.dim() - 4), -4, -1, -3, -2).flatten(-4)


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(int(seed))
    dev = torch.device("cuda")
    heads, kv, dim, page, layers = (case[k] for k in ("heads", "kv", "dim", "page", "layers"))
    length, new = _lengths(case)
    n = len(length)
    rows = n if case["op"] in ("append", "attend") else 2 * n   # forks and compacted copies get rows of their own
    used = -(-length // page)
    columns = int(used.max())
    spare = 3 + (int(used.sum()) if rows > n else 0)
    pages = int(used.sum()) + spare
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    table = torch.full((rows, columns), -1, dtype=torch.int32)
    at = 0
    order_host = order.cpu()
    for i, u in enumerate(used.tolist()):
        table[i, :u] = order_host[at:at + u]
        at += u
    refs = torch.zeros(pages, dtype=torch.int32)
    refs[order_host[:at].long()] = 1
    lens = torch.zeros(rows, dtype=torch.int32)
    lens[:n] = torch.from_numpy(length).int()
    st = {"case": case, "table": table.to(dev), "refs": refs.to(dev), "length": lens.to(dev)}

    if case["op"] in ("append", "attend"):
        codes = torch.empty((pages, layers, 2, kv, page * dim // 2), dtype=torch.uint8, device=dev)
        scales = torch.empty((pages, layers, 2, kv, page, dim // 32), dtype=torch.float16, device=dev)
        # keys have a few large channels, as rotated keys of trained models do; values are even
        weight = torch.randn((kv, 1, dim), generator=g, device=dev).mul(0.5).exp()
        step = max(1, (1 << 27) // (layers * kv * page * dim))
        for a in range(0, pages, step):
            m = min(step, pages - a)
            for which in (0, 1):
                x = torch.randn((m, layers, kv, page, dim), generator=g, device=dev)
                code, d = _quantized(x * weight if which == 0 else x)
                codes[a:a + m, :, which] = _packed_keys(code) if which == 0 else _packed_values(code)
                scales[a:a + m, :, which] = d
        off = np.concatenate([[0], np.cumsum(new)])
        total = int(off[-1])
        st.update(seqs=torch.arange(n, dtype=torch.int32, device=dev),
                  off=torch.from_numpy(off).int().to(dev), total=total, most=int(new.max()), layer=layers - 1,
                  scale=1.0 / math.sqrt(dim))
        dt = DTYPE[case["dtype"]]
        if case["op"] == "append":
            st["k"] = (torch.randn((total, kv, dim), generator=g, device=dev) * weight[:, 0]).to(dt)
            st["v"] = torch.randn((total, kv, dim), generator=g, device=dev).to(dt)
        else:
            st["q"] = (torch.randn((total, heads, dim), generator=g, device=dev) * 1.5).to(dt)
    else:                                                       # bytes are moved, whatever they are
        codes = torch.randint(0, 256, (pages, layers, 2, kv, page * dim // 2), generator=g, device=dev,
                              dtype=torch.uint8)
        scales = torch.rand((pages, layers, 2, kv, page, dim // 32), generator=g, device=dev).half()
        st.update(src=torch.arange(n, dtype=torch.int32, device=dev),
                  dst=torch.arange(n, 2 * n, dtype=torch.int32, device=dev))
        if case["op"] == "compact":
            keep, koff = [], [0]
            for m, k in zip(length.tolist(), _kept(case, length.tolist())):
                at = torch.randperm(m, generator=g, device=dev)[:k].sort().values.int()
                at[:min(4, k)] = torch.arange(min(4, k), device=dev, dtype=torch.int32)
                keep.append(at.sort().values)
                koff.append(koff[-1] + k)
            st.update(keep=torch.cat(keep), keep_off=torch.tensor(koff, dtype=torch.int32, device=dev), total=koff[-1])
    st["codes"], st["scales"] = codes, scales
    return st


# ---------------------------------------------------------------- the plain form

def _new_tokens(st):
    """Of every new token: the number of its sequence in the call, and its position."""
    off = st["off"].long()
    token = torch.arange(st["total"], device=off.device)
    s = torch.searchsorted(off[1:], token, right=True)
    pos = st["length"].long()[st["seqs"].long()[s]] - (off[s + 1] - token)
    return s, pos


def _values(st, which, pages):
    """The values of whole pages: float32 [..., kv, page tokens, D]."""
    case = st["case"]
    dim, page = case["dim"], case["page"]
    c = st["codes"][pages, st["layer"], which]
    nib = torch.stack((c & 15, c >> 4), -1)
    if which == 0:
        nib = nib.unflatten(-2, (page, 4, dim // 32, 4)).transpose(-4, -3)
    else:
        nib = nib.unflatten(-2, (page // 8, 8, 8, dim // 16)).flatten(-2)             # group, c % 8, token, c // 8
        nib = nib.permute(*range(nib.dim() - 4), -4, -2, -1, -3)
    q = nib.reshape(*c.shape[:-1], page, dim // 32, 32).float() - 8
    return (q * st["scales"][pages, st["layer"], which].float().unsqueeze(-1)).flatten(-2)


def _plain_append(st):
    case = st["case"]
    dim, page = case["dim"], case["page"]
    s, pos = _new_tokens(st)
    at = st["table"].long()[st["seqs"].long()[s], pos // page]
    slot = pos % page
    out = []
    for which, x in ((0, st["k"]), (1, st["v"])):
        code, d = _quantized(x.float())
        st["scales"][at, st["layer"], which, :, slot] = d
        codes = st["codes"][:, st["layer"], which]
        if which == 0:
            rows = codes.unflatten(-1, (page, dim // 2))
            rows[at, :, slot] = _packed_keys(code.unsqueeze(-2))
        else:
            units = codes.unflatten(-1, (page // 8, 8, 8, dim // 16))
            w = code.unflatten(-1, (-1, 2, 8))
            units[at, :, slot // 8, :, slot % 8] = (w[..., 0, :] | (w[..., 1, :] << 4)).transpose(-1, -2)
        back = code.float() - 8
        out.append((back.unflatten(-1, (-1, 32)) * d.float().unsqueeze(-1)).flatten(-2))
    return {"k": out[0], "v": out[1]}


def _plain_attend(st):
    case = st["case"]
    heads, kv, dim = case["heads"], case["kv"], case["dim"]
    seqs, most = st["seqs"].long(), st["most"]
    rows = st["table"].long()[seqs].clamp(min=0)
    k = _values(st, 0, rows).transpose(1, 2).flatten(2, 3)      # sequence, kv, token, D
    v = _values(st, 1, rows).transpose(1, 2).flatten(2, 3)
    s, pos = _new_tokens(st)
    at = torch.arange(st["total"], device=s.device) - st["off"].long()[s]
    q = torch.zeros((len(seqs), most, heads, dim), device=s.device)
    q[s, at] = st["q"].float()
    where = torch.full((len(seqs), most), -1, device=s.device)
    where[s, at] = pos
    group = heads // kv
    q = q.unflatten(2, (kv, group)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    score = torch.matmul(q, k.transpose(-1, -2)).mul_(st["scale"]).unflatten(2, (most, group))
    token = torch.arange(k.shape[2], device=s.device)
    p = where[:, :, None]
    seen = token <= p
    if case["window"]:
        seen &= (token > p - case["window"]) | (token < case["sinks"])
    score.masked_fill_(~seen[:, None, :, None, :], -math.inf)
    m = score.amax(-1, keepdim=True)
    e = score.sub_(torch.where(m.isinf(), torch.zeros_like(m), m)).exp_()
    total = e.sum(-1, keepdim=True)
    o = torch.matmul(e.flatten(2, 3), v).unflatten(2, (most, group))
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    o = o.permute(0, 2, 1, 3, 4).flatten(2, 3)
    return {"out": o[s, at].to(DTYPE[case["dtype"]])}


def _plain_release(st, rows):
    """The pages of these rows lose one reader each."""
    page = st["case"]["page"]
    column = torch.arange(st["table"].shape[1], device=rows.device)
    held = column < (-(-st["length"].long()[rows] // page))[:, None]
    ids = st["table"].long()[rows].clamp(min=0)
    st["refs"].index_add_(0, ids.flatten(), -held.flatten().int())


def _plain_fresh(st, need):
    """The lowest-numbered free pages, `need` of them for each entry: [entries][columns], -1 beyond."""
    free = torch.argsort((st["refs"] != 0).int(), stable=True).int()
    first = torch.cumsum(need, 0) - need
    column = torch.arange(st["table"].shape[1], device=need.device)
    some = column < need[:, None]
    got = free[(first[:, None] + column).clamp(max=len(free) - 1)]
    st["refs"].index_add_(0, got.long().flatten(), some.flatten().int())
    return torch.where(some, got, torch.full_like(got, -1))


def _plain_fork(st):
    page = st["case"]["page"]
    src, dst = st["src"].long(), st["dst"].long()
    _plain_release(st, dst)
    n = st["length"].long()[src]
    whole, open_ = n // page, (n % page != 0).long()
    column = torch.arange(st["table"].shape[1], device=src.device)
    shared = column < whole[:, None]
    row = st["table"][src]
    st["refs"].index_add_(0, row.long().clamp(min=0).flatten(), shared.flatten().int())
    fresh = _plain_fresh(st, open_)[:, :1]
    last = (column == whole[:, None]) & (open_ > 0)[:, None]
    st["table"][dst] = torch.where(shared, row, torch.where(last, fresh, torch.full_like(row, -1)))
    st["length"][dst] = n.int()
    some = open_.nonzero()[:, 0]
    a, b = row[some, whole[some]].long(), fresh[some, 0].long()
    st["codes"][b] = st["codes"][a]
    st["scales"][b] = st["scales"][a]
    return _state(st)


def _plain_compact(st):
    case = st["case"]
    page, dim = case["page"], case["dim"]
    src, dst = st["src"].long(), st["dst"].long()
    _plain_release(st, dst)
    off = st["keep_off"].long()
    n = off[1:] - off[:-1]
    fresh = _plain_fresh(st, -(-n // page))
    st["table"][dst] = fresh
    st["length"][dst] = n.int()
    i = torch.arange(st["total"], device=src.device)
    e = torch.searchsorted(off[1:], i, right=True)
    i = i - off[e]
    old = st["keep"].long()
    a, x = st["table"].long()[src[e], old // page], old % page
    b, y = fresh.long()[e, i // page], i % page
    keys = st["codes"][:, :, 0].unflatten(-1, (page, dim // 2))
    keys[b, :, :, y] = keys[a, :, :, x]
    units = st["codes"][:, :, 1].unflatten(-1, (page // 8, 8, 8, dim // 16))
    units[b, :, :, y // 8, :, y % 8] = units[a, :, :, x // 8, :, x % 8]
    st["scales"][b, :, :, :, y] = st["scales"][a, :, :, :, x]
    return _state(st)


def _state(st):
    return {"table": st["table"], "length": st["length"], "refs": st["refs"], "codes": st["codes"],
            "scales": st["scales"].view(torch.int16)}


PLAIN = {"append": _plain_append, "attend": _plain_attend, "fork": _plain_fork, "compact": _plain_compact}


# ---------------------------------------------------------------- one pass

def run(st):
    case = st["case"]
    if not own:
        return PLAIN[case["op"]](st)
    kv = st.get("cache")
    if kv is None:
        from quantized_base_lora_gb300.kvcache import KvCache
        kv = st["cache"] = KvCache(st["codes"], st["scales"], st["table"], st["length"], st["refs"])
    if case["op"] == "append":
        kv.append(st["layer"], st["seqs"], st["off"], st["k"], st["v"])
        k, v = kv.read(st["layer"], st["seqs"], st["off"], st["total"])
        return {"k": k, "v": v}
    if case["op"] == "attend":
        return {"out": kv.attention(st["layer"], st["seqs"], st["off"], st["q"], st["most"], scale=st["scale"],
                                    window=case["window"], sinks=case["sinks"])}
    if case["op"] == "fork":
        kv.fork(st["src"], st["dst"])
    else:
        kv.compact(st["src"], st["dst"], st["keep"], st["keep_off"])
    return _state(st)


# ---------------------------------------------------------------- in 64 bits

def _held_exactly(st, which, seq, n):
    """float64 [kv, n, D]: a sequence's keys or values, each 4-bit field found by its own address."""
    case = st["case"]
    dim, page = case["dim"], case["page"]
    dev = st["codes"].device
    j = torch.arange(n, device=dev)
    slot, c = j % page, torch.arange(dim, device=dev)
    if which == 0:
        byte = slot[:, None] * (dim // 2) + ((c % 32 // 8) * (dim // 32) + c // 32) * 4 + c % 8 // 2
        low = (c % 2 == 0)
    else:
        byte = (slot // 8 * 4 * dim + slot % 8 * (dim // 16))[:, None] + (c % 8) * (dim // 2) + c // 16
        low = (c // 8 % 2 == 0)
    pages = st["table"][seq].long()[j // page]
    field = st["codes"][:, st["layer"], which][pages[:, None], :, byte.expand(n, dim)]      # token, channel, kv
    field = torch.where(low[:, None], field % 16, field // 16).permute(2, 0, 1)
    d = st["scales"][:, st["layer"], which][pages, :, slot].double().transpose(0, 1)
    return (field.double() - 8) * d.repeat_interleave(32, dim=2)


def exact(case, seed):
    if case["op"] not in ("append", "attend"):
        return None                                             # whole numbers only
    st = prepare(case, seed)
    length, new = _lengths(case)
    if case["op"] == "append":
        out = {}
        for name in ("k", "v"):
            x = st[name].double()
            top = x.reshape(*x.shape[:-1], case["dim"] // 32, 32).abs().max(-1).values
            d = (top * 0.125).float().half().double().repeat_interleave(32, dim=-1)
            t = (x / d.clamp(min=1e-30)).nan_to_num(0.0)
            away = torch.sign(t) * torch.floor(t.abs() + 0.5)
            out[name] = away.clamp(-8, 7) * d
        return out
    group = case["heads"] // case["kv"]
    out = torch.zeros((st["total"], case["heads"], case["dim"]), dtype=torch.float64, device="cuda")
    at = 0
    for s, (n, t) in enumerate(zip(length.tolist(), new.tolist())):
        k, v = _held_exactly(st, 0, s, n), _held_exactly(st, 1, s, n)
        j = torch.arange(n, device="cuda")
        for a in range(0, t, 256):
            b = min(t, a + 256)
            p = torch.arange(n - t + a, n - t + b, device="cuda")[:, None]
            dark = j > p
            if case["window"]:
                dark |= (j <= p - case["window"]) & (j >= case["sinks"])
            for h in range(case["heads"]):
                z = st["q"][at + a:at + b, h].double() @ k[h // group].T * st["scale"]
                z[dark] = -math.inf
                out[at + a:at + b, h] = torch.softmax(z, -1) @ v[h // group]
        at += t
    return {"out": out}

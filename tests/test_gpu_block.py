"""Rotary positions, block norms and gated activations on the GPU, against 64 bits."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import block_plain as P  # noqa: E402

if torch.cuda.is_available():
    import quantized_base_lora_gb300 as q
    from quantized_base_lora_gb300 import block as B
    from quantized_base_lora_gb300.kvcache import KvCache

F32, BF16 = torch.float32, torch.bfloat16


def rand(seed, *shape, dtype=F32, scale=1.0):
    g = torch.Generator("cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def close(got, want, allowed, dtype):
    """Within the allowed distance, and half a step of the output."""
    off = (got.double() - want).abs()
    room = allowed + want.abs() * P.HALF[dtype] * 1.001
    assert got.dtype == dtype and torch.isfinite(got).all()
    assert (off <= room).all(), float((off / room.clamp(min=1e-300)).max())


# ---------------------------------------------------------------- rotary positions

def check_rope(rope, case, pos, x, y):
    w, size = case
    want, mag = P.rope(x.double(), pos, w, size, rope)
    assert ((y.double() - want).abs() <= P.rope_allowed(want, mag, y.dtype)).all()
    passed = mag.sum((0, 1)) == 0
    assert torch.equal(y[..., passed], x[..., passed].to(y.dtype))


@pytest.mark.parametrize("layout", ["half", "pairs"])
@pytest.mark.parametrize("dim,rot,heads,kv", [(128, 128, 4, 1), (128, 64, 3, 3), (64, 64, 1, 0), (256, 256, 2, 1),
                                             (96, 40, 5, 2), (80, 34, 2, 1), (6, 2, 7, 3), (512, 512, 1, 1), (8, 8, 1, 1)])
@pytest.mark.parametrize("tokens,dtype,out", [(1, F32, BF16), (7, BF16, BF16), (33, F32, F32), (5, BF16, F32)])
def test_rotations(layout, dim, rot, heads, kv, tokens, dtype, out):
    rope = B.Rope(dim, rot, layout, base=500000.0)
    pos = torch.randint(0, 1 << 20, (tokens,), device="cuda", dtype=torch.int32,
                        generator=torch.Generator("cuda").manual_seed(dim + rot))
    qk = rand(dim, tokens, heads + kv, dim, dtype=dtype, scale=3.0)
    x, k = qk[:, :heads], qk[:, heads:]
    got = rope(pos, x, k if kv else None, dtype=out)
    for have, src in zip(got if kv else (got,), (x, k)):
        assert have.is_contiguous()
        check_rope(layout, P.frequencies(rot, 500000.0), pos, src, have)


@pytest.mark.parametrize("layout", ["half", "pairs"])
@pytest.mark.parametrize("dtype,out", [(BF16, BF16), (F32, F32), (F32, BF16), (BF16, F32)])
@pytest.mark.parametrize("dim,rot,heads,kv", [(80, 34, 30, 3), (80, 80, 35, 1), (66, 66, 9, 2), (64, 64, 5, 0)])
def test_rotations_of_many_tokens(layout, dtype, out, dim, rot, heads, kv):
    """Several heads a thread, the last of them not full; queries and keys in tensors of their own."""
    rope, tokens = B.Rope(dim, rot, layout), 2503
    pos = torch.randint(0, 1 << 17, (tokens,), device="cuda", dtype=torch.int32, generator=torch.Generator("cuda").manual_seed(dim))
    x, k = rand(1, tokens, heads, dim, dtype=dtype), rand(2, tokens, kv, dim, dtype=dtype)
    got = rope(pos, x, k if kv else None, dtype=out)
    for have, src in zip(got if kv else (got,), (x, k)):
        check_rope(layout, P.frequencies(rot, 10000.0), pos, src, have)


@pytest.mark.parametrize("scaling,factor,original,magnitude", [
    ("linear", 4.0, 0, None), ("base", 8.0, 0, None), ("bands", 8.0, 8192, None), ("ramp", 16.0, 4096, None),
    ("ramp", 16.0, 4096, 1.0), (None, 1.0, 0, 0.25)])
def test_scalings_at_far_positions(scaling, factor, original, magnitude):
    rope = B.Rope(128, layout="half", scaling=scaling, factor=factor, original=original, magnitude=magnitude)
    pos = ints(0, 1, 4095, 131071, 1 << 24, (1 << 31) - 1, -1, -(1 << 31), 987654321)
    x = rand(3, len(pos), 2, 128)
    w, size = P.frequencies(128, 10000.0, scaling, factor, original)
    # the plan's frequencies are held to 2^-65 of a turn and 2^-46 of themselves (the CPU test), which 2^31 positions
    # make 2^-15 radians of; the rotation itself is compared with what the plan holds
    held = [t / 2.0 ** 64 * math.tau for t in list(rope.plan.turn)[:64]]
    assert max(abs(a / b - 1) for a, b in zip(held, w)) < 2.0 ** -40
    want, mag = P.rope(x.double(), torch.zeros_like(pos), held, 1.0, "half")
    turns = torch.tensor([[(int(p) * t % 2 ** 64) / 2.0 ** 64 for t in list(rope.plan.turn)[:64]] for p in pos.tolist()],
                         dtype=torch.float64, device="cuda") * math.tau
    size = size if magnitude is None else magnitude
    cos, sin = turns.cos()[:, None] * size, turns.sin()[:, None] * size
    a, b = x.double()[..., :64], x.double()[..., 64:]
    want = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    assert ((rope(pos, x).double() - want).abs() <= P.rope_allowed(want, mag * size, F32)).all()


def test_rotation_in_place_strided_and_at_odd_addresses():
    rope = B.Rope(64, 48, "half")
    pos = ints(*range(100, 109))
    flat = rand(5, 9 * 400 + 3)
    for shift, step in ((0, 400), (1, 399), (3, 5 * 64)):
        wide = flat[shift:shift + 9 * step].clone().view(9, step) if shift == 0 else \
            torch.as_strided(flat.clone(), (9, step), (step, 1), shift)
        before = wide.clone()
        x, k = wide[:, :3 * 64].view(9, 3, 64), wide[:, 3 * 64:5 * 64].view(9, 2, 64)
        out = torch.full((9, 6, 64), 7.0, device="cuda")
        apart = rope(pos, x, k, q_out=out[:, :3], k_out=out[:, 4:])
        assert (out[:, 3] == 7).all()
        assert torch.equal(wide, before)
        rope(pos, x, k, q_out=x, k_out=k)
        assert torch.equal(x, apart[0]) and torch.equal(k, apart[1])
        assert torch.equal(wide[:, 5 * 64:], before[:, 5 * 64:])
        check_rope("half", P.frequencies(48), pos, before[:, :3 * 64].view(9, 3, 64), x)


def test_many_rotations_and_few_are_alike():
    """The kernels for few and many tokens, and for wide and single accesses, on the same values."""
    for dim in (128, 6):
        rope = B.Rope(dim, layout="pairs")
        n = 3000 if dim == 128 else 40000
        pos = torch.arange(n, device="cuda", dtype=torch.int32)
        x = rand(9, n, 9, dim, dtype=BF16)
        many = rope(pos, x)
        some = torch.cat([rope(pos[a:a + 7], x[a:a + 7]) for a in (0, 1000, n - 7)])
        assert torch.equal(some, torch.cat([many[a:a + 7] for a in (0, 1000, n - 7)]))
        check_rope("pairs", P.frequencies(dim), pos[-7:], x[-7:], many[-7:])


def test_rotation_of_no_tokens_and_of_values_out_of_the_ordinary():
    rope = B.Rope(64)
    assert rope(ints(), torch.empty((0, 2, 64), device="cuda")).shape == (0, 2, 64)
    x = rand(1, 3, 2, 64)
    x[1, 0, 5], x[1, 1, 7] = math.nan, math.inf
    y = rope(ints(1, 2, 3), x)
    bad = ~torch.isfinite(y)
    want = torch.zeros_like(bad)
    want[1, 0, [5, 37]], want[1, 1, [7, 39]] = True, True
    assert torch.equal(bad, want)                        # the pairs that hold them, and no other


def test_positions_of_a_batch():
    c = KvCache.allocate(n_pages=32, page_tokens=16, n_layers=1, n_kv_heads=1, head_dim=64, max_seqs=4, max_pages=8)
    c.extend(ints(2, 0), ints(0, 30, 37))
    assert c.positions(ints(2, 0), ints(0, 30, 37), 37).tolist() == list(range(30)) + list(range(7))
    c.extend(ints(0, 2), ints(0, 1, 4))
    assert c.positions(ints(0, 2), ints(0, 1, 4), 4).tolist() == [7, 30, 31, 32]
    assert c.positions(ints(1), ints(0, 0), 0).tolist() == []
    c.check()
    assert c.positions(ints(), ints(0), 3).tolist() == [-1] * 3
    assert c.positions(ints(0, 2), ints(0, 1, 4), 6).tolist() == [7, 30, 31, 32, -1, -1]      # a padded call
    with pytest.raises(q.OvlError) as e:
        c.check()
    assert e.value.status == q.OVL_E_ARG
    assert c.positions(ints(9), ints(0, 2), 2).tolist() == [-1, -1]
    with pytest.raises(q.OvlError):
        c.check()
    assert c.positions(ints(1), ints(0, 2), 2).tolist() == [-1, -1]      # a row that holds less than its new tokens
    c.check()


# ---------------------------------------------------------------- block norms

def check_norm(x, y, pre, post, gate, row, alpha, beta, got, h_dtype):
    z, off = P.normed(y.double(), post.kind if post else None, *((post.weight, post.bias, post.eps, post.offset) if post else
                                                                 (None, None, 0, 0))) if y is not None else (None, 0)
    want = alpha * x.double()
    room = 2.0 ** -23 * want.abs()
    if y is not None:
        g = torch.ones_like(z) if gate is None else gate.double()[row.long()] if row is not None else \
            gate.double().expand_as(z) if gate.dim() == 1 or len(gate) in (1, len(z)) else None
        want = want + beta * g * z
        room = room + (abs(beta) * g.abs() * (off + 2.0 ** -22 * z.abs()) + 2.0 ** -23 * want.abs())
    xs, h = got
    close(xs, want, room, x.dtype)
    if pre is None:
        assert h is None
        return
    out, off = P.normed(want, pre.kind, pre.weight, pre.bias, pre.eps, pre.offset)
    # what x' may be off by goes through the norm: times r and the weight, and by the root of the row's mean square
    # into r; by the mean into every element
    c = want - want.mean(-1, keepdim=True) * (pre.kind == "layer")
    r = 1 / torch.sqrt(c.square().mean(-1, keepdim=True) + pre.eps)
    w = torch.ones_like(want) if pre.weight is None else (pre.weight.double() + pre.offset).expand_as(want)
    spread = room.square().mean(-1, keepdim=True).sqrt()
    close(h, out, off + w.abs() * r * (room + spread * (1 + (c * r).abs())), h_dtype)


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("post_kind", [None, "rms", "layer"])
@pytest.mark.parametrize("hidden", [1, 7, 64, 96, 1000, 1024, 1155, 2047, 4096, 5120, 8192, 9001, 16384])
def test_norms(kind, post_kind, hidden):
    for tokens, xd, yd, hd in ((1, BF16, F32, BF16), (5, F32, BF16, F32)):
        x, y = rand(hidden, tokens, hidden, dtype=xd) + 0.5, rand(hidden + 1, tokens, hidden, dtype=yd, scale=2.0)
        wd = BF16 if tokens == 1 else F32
        pre = B.Norm(kind, rand(2, hidden, dtype=wd), rand(3, hidden, dtype=wd) if tokens == 5 else None, 1e-5, 1.0)
        post = B.Norm(post_kind, rand(4, hidden, dtype=wd), rand(5, hidden, dtype=wd), 1e-6, 0.0) if post_kind else None
        gate = rand(6, tokens, hidden) if tokens == 5 else None
        n = B.BlockNorm(hidden, pre, post, alpha=0.75, beta=1.5)
        check_norm(x, y, pre, post, gate, None, 0.75, 1.5, n(x, y, gate=gate, dtype=hd), hd)


@pytest.mark.parametrize("xd", [F32, BF16])
@pytest.mark.parametrize("yd", [F32, BF16])
@pytest.mark.parametrize("hd", [F32, BF16])
@pytest.mark.parametrize("hidden", [512, 4096, 8192, 1001, 5001])
def test_norm_types_over_more_rows_than_fit_at_once(xd, yd, hd, hidden):
    tokens = 1700 if hidden < 5000 else 700
    x, y = rand(1, tokens, hidden, dtype=xd), rand(2, tokens, hidden, dtype=yd)
    pre, post = B.Norm("rms", rand(3, hidden)), B.Norm("rms", rand(4, hidden))
    n = B.BlockNorm(hidden, pre, post)
    xs, h = n(x, y, dtype=hd)
    some = torch.tensor([0, 1, 303, 304, 607, 608, tokens // 2, tokens - 1], device="cuda")
    check_norm(x[some], y[some], pre, post, None, None, 1.0, 1.0, (xs[some], h[some]), hd)
    # a row's bits do not depend on the rows beside it
    one = n(x[tokens - 1:], y[tokens - 1:], dtype=hd)
    assert torch.equal(one[0][0], xs[-1]) and torch.equal(one[1][0], h[-1])


@pytest.mark.parametrize("xd", [F32, BF16])
@pytest.mark.parametrize("hidden", [3, 100, 160, 161, 320, 333, 640, 641, 1283, 2049, 4099,           # element by element, but for 160, 320, 640
                                    8, 128, 256, 264, 512, 520, 1032, 1536, 2048, 2056])
def test_gated_rows_of_every_width(xd, hidden):
    """Several rounds of rows, the last one not full; layer norms, biases and a gate for each of five sequences."""
    tokens = 5003 if hidden < 700 else 1301
    yd, wd = (BF16, F32) if xd == F32 else (F32, BF16)
    x, y, gate = rand(1, tokens, hidden, dtype=xd), rand(2, tokens, hidden, dtype=yd), rand(3, 5, hidden, dtype=wd)
    row = torch.randint(0, 5, (tokens,), generator=torch.Generator().manual_seed(4)).int().cuda()
    pre = B.Norm("layer", rand(5, hidden, dtype=wd), rand(6, hidden, dtype=wd))
    post = B.Norm("layer", rand(7, hidden, dtype=wd), rand(8, hidden, dtype=wd), 1e-3, 1.0)
    n = B.BlockNorm(hidden, pre, post, alpha=0.5, beta=2.0)
    xs, h = n(x, y, gate=gate, gate_row=row, dtype=xd)
    check_norm(x, y, pre, post, gate, row, 0.5, 2.0, (xs, h), xd)
    for t in (0, tokens - 1):                            # alone, the same bits
        one = n(x[t:t + 1], y[t:t + 1], gate=gate, gate_row=row[t:t + 1], dtype=xd)
        assert torch.equal(one[0][0], xs[t]) and torch.equal(one[1][0], h[t])


@pytest.mark.parametrize("hidden", [256, 255, 12288])
def test_gates_of_rows(hidden):
    """A row of -1 (or beyond the gates) leaves the block's output out, whatever it holds."""
    tokens = 9
    x, y, gate = rand(1, tokens, hidden), rand(2, tokens, hidden), rand(3, 3, hidden, dtype=BF16)
    row = ints(0, 2, -1, 1, 3, 0, 2, 1 << 30, 1)
    out = (row < 0) | (row > 2)
    y[out] = math.nan
    n = B.BlockNorm(hidden, B.Norm("layer"), B.Norm("layer"), alpha=2.0)
    xs, h = n(x, y, gate=gate, gate_row=row)
    assert torch.equal(xs[out], 2 * x[out])
    check_norm(x[~out], y[~out], n.pre, n.post, gate, row[~out], 2.0, 1.0, (xs[~out], h[~out]), F32)
    check_norm(x[out], None, n.pre, None, None, None, 2.0, 1.0, (xs[out], h[out]), F32)
    for g in (gate[0], gate[:1]):                        # one gate for all
        check_norm(x[~out], y[~out], n.pre, n.post, g, None, 2.0, 1.0, n(x[~out], y[~out], gate=g), F32)


@pytest.mark.parametrize("hidden,shift,step", [(512, 0, 1024), (512, 4, 520), (500, 0, 512), (77, 1, 101)])
def test_norms_in_place_strided_and_at_odd_addresses(hidden, shift, step):
    tokens = 21
    flat = rand(7, tokens * step + 8)
    x = torch.as_strided(flat, (tokens, hidden), (step, 1), shift)
    y = rand(8, tokens, hidden)
    pre = B.Norm("rms", rand(9, hidden + 1)[1:])         # a weight at an odd address too
    n = B.BlockNorm(hidden, pre)
    want = n(x.clone(), y)
    before = flat.clone()
    back = torch.full((tokens, hidden + 8), 3.0, device="cuda")
    got = n(x, y, x_out=x, h_out=back[:, :hidden])
    assert got[0] is x and torch.equal(x, want[0]) and torch.equal(got[1], want[1])
    assert (back[:, hidden:] == 3).all()
    mask = torch.ones_like(flat, dtype=torch.bool)
    torch.as_strided(mask, (tokens, hidden), (step, 1), shift).fill_(False)
    assert torch.equal(flat[mask], before[mask])
    check_norm(torch.as_strided(before, (tokens, hidden), (step, 1), shift), y, pre, None, None, None, 1.0, 1.0, got, F32)


def test_norm_without_a_block_output_or_a_next_block():
    x, y = rand(1, 4, 640, dtype=BF16), rand(2, 4, 640)
    n = B.BlockNorm(640, B.Norm("rms"))
    check_norm(x, None, n.pre, None, None, None, 1.0, 1.0, n(x, dtype=F32), F32)
    m = B.BlockNorm(640, None, B.Norm("rms", eps=1e-3))
    check_norm(x, y, None, m.post, None, None, 1.0, 1.0, m(x, y), BF16)
    zero = torch.zeros((2, 640), device="cuda")
    assert (n(zero)[1] == 0).all()                       # eps keeps the root from zero
    empty = n(x[:0], y[:0])
    assert empty[0].shape == empty[1].shape == (0, 640)


def test_statistics_of_a_large_mean():
    """A mean far above the spread: squares around it, not a difference of two sums."""
    x = rand(1, 3, 4096) + 1000.0
    n = B.BlockNorm(4096, B.Norm("layer", eps=0.0))
    want, _ = P.normed(x.double(), "layer", None, None, 0.0, 0.0)
    # the mean, 1000, is off by 2^-19 of itself at most
    assert (n(x)[1].double() - want).abs().max() < 1000 * 2.0 ** -19 * 1.1


# ---------------------------------------------------------------- gated activations

@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "relu"])
@pytest.mark.parametrize("tokens,width,dtype,out", [(1, 14336, F32, BF16), (3, 1, F32, F32), (5, 333, BF16, BF16),
                                                    (64, 96, BF16, F32), (2, 4097, F32, F32)])
def test_activations(act, tokens, width, dtype, out):
    gate, up = rand(width, tokens, width, dtype=dtype, scale=4.0), rand(width + 1, tokens, width, dtype=dtype)
    got = B.glu(gate, up, act=act, dtype=out)
    g, u = gate.double(), up.double()
    # e^-v and erf to 2 ulp, of an argument that is off by up to 5 roundings of 2^-24 (a tenth of 100 at the most where
    # what follows is not below 2^-24 of v), a quotient to 2 ulp: 2^-20 of |v u|
    close(got, P.activated(g, act) * u, 2.0 ** -20 * (g * u).abs(), out)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("tokens,width", [(70000, 3), (301, 1023), (301, 1025), (77, 5001)])
def test_activations_of_odd_halves(dtype, tokens, width):
    """Gate and up side by side at an odd width: rows begin at any address."""
    both = rand(width, tokens, 2 * width, dtype=dtype)
    gate, up = both[:, :width], both[:, width:]
    back = torch.full((tokens, width + 2), 3.0, device="cuda", dtype=dtype)
    B.glu(gate, up, act="gelu_tanh", out=back[:, :width])
    g, u = gate.double(), up.double()
    close(back[:, :width], P.activated(g, "gelu_tanh") * u, 2.0 ** -20 * (g * u).abs(), dtype)
    assert (back[:, width:] == 3).all()
    B.glu(gate, up, act="gelu_tanh", out=gate)           # in place
    assert torch.equal(gate, back[:, :width])


def test_activations_in_place_strided_and_of_large_values():
    both = rand(1, 6, 2 * 200)                           # gate and up of one projection, side by side
    gate, up = both[:, :200], both[:, 200:]
    want = B.glu(gate, up)
    B.glu(gate, up, out=up)
    assert torch.equal(up, want)
    odd = rand(2, 6, 2 * 99 + 1)
    want = B.glu(odd[:, :99].contiguous(), odd[:, 100:].contiguous())
    assert torch.equal(B.glu(odd[:, :99], odd[:, 100:]), want)
    v = torch.tensor([[100.0, -100.0, 1e30, -1e30, 0.0, math.nan, 88.5, -88.5]], device="cuda")
    one = torch.ones_like(v)
    for act in ("silu", "gelu", "gelu_tanh", "relu"):
        got = B.glu(v, one, act=act)[0]
        assert got[0] == 100 and got[2] == 1e30 and got[4] == 0 and got[5].isnan()
        assert (got[[1, 3, 7]].abs() < 1e-30).all() and got[6] == 88.5
    assert B.glu(v[:0], v[:0]).shape == (0, 8)


# ---------------------------------------------------------------- streams, graphs, devices

def test_on_another_stream_and_in_a_graph():
    x, y, w = rand(1, 16, 768, dtype=BF16), rand(2, 16, 768), rand(3, 768)
    n = B.BlockNorm(768, B.Norm("rms", w))
    rope, pos = B.Rope(64), torch.arange(16, device="cuda", dtype=torch.int32)

    def step():
        xs, h = n(x, y, dtype=F32)
        r = rope(pos, h.view(16, 12, 64))
        return xs, r, B.glu(r.flatten(1), y)

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for seed in (5, 6):                                  # replays read what is there then
        x.copy_(rand(seed, 16, 768))
        pos.add_(1000)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, step()))


def test_what_the_torch_side_refuses():
    x, w = torch.zeros((4, 64), device="cuda"), torch.ones(64, device="cuda")
    n = B.BlockNorm(64, B.Norm("rms", w))
    rope = B.Rope(64)
    h = x.view(4, 1, 64)
    for call in (lambda: n(x.half()), lambda: n(x[:, :32]), lambda: n(x, x[:3]), lambda: n(x.T), lambda: n(x, dtype=torch.float16),
                 lambda: n(x, gate=x), lambda: n(x, x, gate=x[:3]), lambda: n(x, x, gate=x, gate_row=ints(0)),
                 lambda: n(x, x, gate_row=ints(0, 0, 0, 0)), lambda: n(x, x, gate=x[:0]), lambda: n(x, x_out=x.bfloat16()),
                 lambda: n(x, h_out=x[:2]), lambda: B.BlockNorm(64, None)(x, h_out=x), lambda: n(x, x.cpu()),
                 lambda: B.BlockNorm(64, B.Norm("rms", w[:3])), lambda: B.BlockNorm(64, B.Norm("rms", w, w.bfloat16())),
                 lambda: rope(ints(0, 1, 2), h), lambda: rope(torch.zeros(4, device="cuda"), h), lambda: rope(ints(0, 1, 2, 3), x),
                 lambda: rope(ints(0, 1, 2, 3), h, h.bfloat16()), lambda: rope(ints(0, 1, 2, 3), h, k_out=h),
                 lambda: rope(ints(0, 1, 2, 3), h, dtype=BF16, q_out=h), lambda: rope(ints(0, 1, 2, 3), h.transpose(0, 2)),
                 lambda: B.glu(x, x[:2]), lambda: B.glu(x, x.bfloat16()), lambda: B.glu(x, x, act="tanh"),
                 lambda: B.glu(x, x, out=x[:1]), lambda: B.glu(h, h)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(q.OvlError):                      # tokens that overlap
        rope(ints(0, 1, 2, 3), h, q_out=torch.as_strided(torch.zeros(64, device="cuda"), (4, 1, 64), (0, 64, 1)))


def test_rotations_of_many_heads_and_tokens():
    rope = B.Rope(64, 48, "pairs")
    pos = torch.arange(4001, device="cuda", dtype=torch.int32) * 31
    qk = rand(4, 4001, 45, 64, dtype=BF16)
    q2, k2 = rope(pos, qk[:, :36], qk[:, 36:], dtype=F32)
    for a, b in ((qk[:, :36], q2), (qk[:, 36:], k2)):
        check_rope("pairs", P.frequencies(48), pos, a, b)


def tail(act, until):
    """Negative gates down to `until`, densely, beside ups of several sizes; the result in 64 bits."""
    gate = -torch.linspace(0.01, until, 4096, device="cuda").expand(3, 4096).contiguous()
    up = torch.tensor([1.0, -3e5, 2e-3], device="cuda")[:, None].expand(3, 4096).contiguous()
    v = gate.double()                                    # ndtr ends at 0 below -8.3: by erfc here
    return gate, up, (v / 2 * torch.erfc(-v / math.sqrt(2)) if act == "gelu" else P.activated(v, act)) * up.double()


@pytest.mark.parametrize("out", [F32, BF16])
def test_the_negative_tail_of_gelu(out):
    """Relative to the result, which is far below |v u| there.  The argument of erfc is off by two roundings, 2^-23 of
    it, which a slope of up to v^2 + 1 multiplies; erfc itself 4 ulp, 2^-21; two products: (v^2 + 6) 2^-23."""
    gate, up, want = tail("gelu", 12.5)
    close(B.glu(gate, up, act="gelu", dtype=out), want, (gate.double().square() + 6) * 2.0 ** -23 * want.abs(), out)


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("out", [F32, BF16])
def test_the_negative_tail_of_the_sigmoids(act, out):
    """Relative to the result: e^ to 2 ulp of an argument that is off by five roundings (gelu_tanh; silu's is exact),
    2^-21 of it, a sum, a quotient to 2 ulp and a product: 2^-20 more.  Below 2^-119 the activation may be 0."""
    gate, up, want = tail(act, 104.0 if act == "silu" else 10.6)
    v = gate.double()
    slope = 2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3).abs() if act == "gelu_tanh" else 0.0
    close(B.glu(gate, up, act=act, dtype=out), want, (slope * 2.0 ** -21 + 2.0 ** -20) * want.abs() + 2.0 ** -119 * up.double().abs(), out)

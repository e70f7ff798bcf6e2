"""A decoder block's step as it is used: norms, projections, rotary positions, cache, attention, activation and experts
one behind the other, each stage against 64 bits on what the stage before gave it; and the same step captured."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import block_plain as P  # noqa: E402
import oracle as O  # noqa: E402
import synth as S  # noqa: E402
from test_gpu_block import check_norm, close, ints, rand  # noqa: E402

if torch.cuda.is_available():
    import quantized_base_lora_gb300 as q
    from quantized_base_lora_gb300 import block as B
    from quantized_base_lora_gb300.kvcache import KvCache
    from quantized_base_lora_gb300.runtime import Runtime

HIDDEN, HEADS, KV, DIM, FFN, EXPERTS = 256, 4, 2, 64, 512, 6
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def block():
    rng = np.random.default_rng(3)
    shapes = [(HEADS * DIM, HIDDEN), (KV * DIM, HIDDEN), (KV * DIM, HIDDEN), (HIDDEN, HEADS * DIM), (FFN, HIDDEN),
              (FFN, HIDDEN), (HIDDEN, FFN), (EXPERTS * FFN, HIDDEN), (EXPERTS * FFN, HIDDEN), (EXPERTS * HIDDEN, FFN)]
    base = S.build_base(S.Q4_0, [(0, i, S.gaussian(rng, s, 0.06)) for i, s in enumerate(shapes)])
    rt = Runtime(arena_bytes=32 << 20)
    q.check(rt.load_base(base.quant, [(t.layer, t.proj, t.d_out, t.d_in, t.qs_off, t.d_off) for t in base.tensors],
                         base.buf, S.content_digest(base.buf)), rt.ctx)
    w = [torch.from_numpy(np.asarray(O.dequantize(S.Q4_0, *p), np.float64)).cuda() for p in base.planes]
    yield rt, w
    rt.close()


def test_a_prompt_and_decode_steps(block):
    rt, w = block
    cache = KvCache.allocate(n_pages=32, page_tokens=16, n_layers=1, n_kv_heads=KV, head_dim=DIM, max_seqs=3, max_pages=8)
    rope = B.Rope(DIM, 48, "half", scaling="linear", factor=2.0)
    pre, post = B.Norm("rms", rand(1, HIDDEN), eps=1e-5), B.Norm("layer", rand(2, HIDDEN), rand(3, HIDDEN))
    first, second, last = B.BlockNorm(HIDDEN, pre), B.BlockNorm(HIDDEN, pre, post, beta=0.5), B.BlockNorm(HIDDEN, None)
    moe = B.Moe.from_base(rt, 7, 8, 9, EXPERTS, 2, router=rand(4, EXPERTS, HIDDEN) * 0.1, max_tokens=64)
    gate = rand(5, 3, HIDDEN)

    def projected(i, h):
        y = rt.forward(i, h)
        want = h.double() @ w[i].T
        # the projections' own bound
        assert ((y.double() - want).abs() <= 2e-3 * (h.double().abs() @ w[i].abs().T) + 1e-5).all()
        return y

    have = [0, 0, 0]
    for rows, counts in (([0, 2], [37, 5]), ([2, 0, 1], [1, 1, 11]), ([0, 1, 2], [1, 1, 1])):
        n, off, seqs = sum(counts), ints(*np.concatenate([[0], np.cumsum(counts)]).tolist()), ints(*rows)
        x = rand(n, n, HIDDEN, dtype=BF16)
        row = torch.repeat_interleave(seqs, torch.tensor(counts, device="cuda"))
        cache.extend(seqs, off)
        pos = cache.positions(seqs, off, n)
        assert pos.tolist() == [have[r] + i for r, c in zip(rows, counts) for i in range(c)]
        x, h = first(x)
        check_norm(x, None, pre, None, None, None, 1.0, 1.0, (x, h), BF16)
        qry, key, val = (projected(i, h).unflatten(-1, (-1, DIM)) for i in range(3))
        q2, k2 = rope(pos, qry, key, dtype=BF16)
        for a, b in ((qry, q2), (key, k2)):
            want, mag = P.rope(a.double(), pos, *P.frequencies(48, scaling="linear", factor=2.0), "half")
            assert ((b.double() - want).abs() <= P.rope_allowed(want, mag, BF16)).all()
        cache.append(0, seqs, off, k2, val.bfloat16())
        o = cache.attention(0, seqs, off, q2, max(counts))
        at = 0
        for r, c in zip(rows, counts):
            have[r] += c
            k, v = (t.double().repeat_interleave(HEADS // KV, 1) for t in cache.read(0, ints(r), ints(0, have[r]), have[r]))
            s = torch.einsum("ihd,jhd->hij", q2[at:at + c].double(), k) / math.sqrt(DIM)
            s.masked_fill_(torch.arange(have[r], device="cuda") > pos[at:at + c, None], -math.inf)
            want = torch.einsum("hij,jhd->ihd", s.softmax(-1), v)
            # bf16: half a step, and weights to 11 bits with 32-bit scores: 2^-9 of the values
            assert ((o[at:at + c].double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -9 * v.abs().max()).all()
            at += c
        y = projected(3, o.flatten(1))
        x2, h = second(x, y, gate=gate, gate_row=row.int())
        check_norm(x, y, pre, post, gate, row, 1.0, 0.5, (x2, h), BF16)
        g, u = projected(4, h), projected(5, h)
        a = B.glu(g, u, dtype=BF16)
        close(a, P.activated(g.double(), "silu") * u.double(), 2.0 ** -20 * (g.double() * u.double()).abs(), BF16)
        x3, h = second(x2, projected(6, a))
        y, choice, weight = moe(h, routing=True)
        want, room = P.moe(h.double().cpu(), *(t.cpu().unflatten(0, (EXPERTS, -1)) for t in w[7:]), choice.cpu(),
                           weight.double().cpu(), "silu", False)
        close(y, want.cuda(), room.cuda(), BF16)
        x4, none = last(x3, y)
        assert none is None
        close(x4, x3.double() + y.double(), 2.0 ** -22 * (x3.double().abs() + y.double().abs()), BF16)
    cache.check()
    q.check(rt.check_device(), rt.ctx)


def test_a_captured_step_reads_lengths_and_positions_on_the_device(block):
    """Replays of one graph: every step takes the next positions, as the cache's lengths have them then."""
    rt, _ = block
    rope, norm = B.Rope(DIM), B.BlockNorm(HIDDEN, B.Norm("rms"))
    moe = B.Moe.from_base(rt, 7, 8, 9, EXPERTS, 2, router=rand(4, EXPERTS, HIDDEN), max_tokens=8)
    seqs, off = ints(1, 0), ints(0, 1, 2)
    x, y = rand(1, 2, HIDDEN, dtype=BF16), rand(2, 2, HIDDEN)

    def fresh():
        return KvCache.allocate(n_pages=8, page_tokens=16, n_layers=1, n_kv_heads=HEADS, head_dim=DIM, max_seqs=2, max_pages=4)

    def step(c):
        c.extend(seqs, off)
        xs, h = norm(x, y)
        qk = h.view(2, HEADS, DIM)
        r, k = rope(c.positions(seqs, off, 2), qk, qk)
        c.append(0, seqs, off, k, qk)
        return moe(c.attention(0, seqs, off, r, 1).flatten(1))

    a = fresh()
    want = []
    for _ in range(20):
        want.append(step(a).clone())
    b = fresh()
    step(b)                                              # first calls outside of the capture
    b.release(seqs)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step(b)
    for i in range(20):
        g.replay()
        assert torch.equal(out, want[i])
    assert b.length.tolist() == [20, 20]
    a.check()
    b.check()

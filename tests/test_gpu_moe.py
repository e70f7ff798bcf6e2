"""The mixture-of-experts layer on the GPU, against 64 bits."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import block_plain as P  # noqa: E402
import oracle as O  # noqa: E402
import synth as S  # noqa: E402

if torch.cuda.is_available():
    import quantized_base_lora_gb300 as q
    from quantized_base_lora_gb300 import block as B

F32, BF16 = torch.float32, torch.bfloat16
QUANTS = [O.Q8_0, O.Q4_0, O.Q4_K]


def rand(seed, *shape, dtype=F32, scale=1.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * scale).to(dtype).cuda()


class Layer:
    def __init__(self, quant, n, hidden, ffn, top, seed=0, router=True, **kw):
        rng = np.random.default_rng(seed)
        made = [P.experts(rng, quant, n, r, c) for r, c in ((ffn, hidden), (ffn, hidden), (hidden, ffn))]
        self.w = [w for _, w in made]
        planes = [tuple(torch.from_numpy(p).cuda() for p in planes) for planes, _ in made]
        self.router = rand(seed + 1, n, hidden, scale=2 / math.sqrt(hidden), dtype=kw.pop("router_dtype", F32)) if router else None
        self.act = kw.get("act", "silu")
        self.moe = B.Moe(quant, n, hidden, ffn, *planes, top_k=top, router=self.router, **kw)

    def check(self, x, y, choice, weight):
        f32 = x.dtype == F32
        want, room = P.moe(x.double().cpu(), *self.w, choice.cpu(), weight.double().cpu(), self.act, f32)
        got = y.double().cpu()
        assert y.dtype == x.dtype and torch.isfinite(got).all()
        off = (got - want).abs()
        room = room + want.abs() * P.HALF[x.dtype] * 1.001
        assert (off <= room).all(), float((off / room.clamp(min=1e-300)).max())
        # and in the mean square, where the roundings do not add up: 2^-18 of an fp32 output, half a step of a bf16 one
        mean = want.square().mean(-1).sqrt()
        assert (off.square().mean(-1).sqrt() <= mean * (2.0 ** -18 if f32 else 2.0 ** -8) + 1e-300).all()


@pytest.mark.parametrize("quant", QUANTS, ids=["q8_0", "q4_0", "q4_K"])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("n,top,hidden,ffn,tokens", [
    (8, 2, 256, 512, 1), (8, 2, 512, 256, 2), (4, 4, 256, 256, 9), (16, 3, 768, 256, 40), (1, 1, 256, 256, 17),
    (512, 16, 256, 256, 3), (60, 5, 1280, 512, 64), (3, 2, 256, 1024, 128)])
def test_layers(quant, dtype, n, top, hidden, ffn, tokens):
    L = Layer(quant, n, hidden, ffn, top, seed=n, max_tokens=tokens)
    x = rand(7, tokens, hidden, dtype=dtype)
    y, choice, weight = L.moe(x, routing=True)
    c, w, gap = P.route(x.cpu(), L.router.cpu(), None, "softmax", top, True, 1.0)
    assert gap > 1e-5                                    # 2^-19 of scores of a few units; no choice is that close here
    assert torch.equal(choice.cpu(), c)
    assert (weight.cpu().double() - w).abs().max() < 2.0 ** -18
    L.check(x, y, c, w)
    assert torch.equal(L.moe(x), y)                      # the same call, the same bits


@pytest.mark.parametrize("quant", [O.Q8_0, O.Q4_0], ids=["q8_0", "q4_0"])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("hidden,ffn", [(32, 32), (64, 96), (96, 64), (160, 32), (288, 224), (544, 800), (1056, 352)])
def test_odd_sizes(quant, dtype, hidden, ffn):
    """Rows whose scales begin at any even address, last stages of 1 to 7 blocks, tiles of half a block."""
    L = Layer(quant, 5, hidden, ffn, 2, seed=hidden, router=False, max_tokens=20)
    for tokens in (1, 20):
        x = rand(3, tokens, hidden, dtype=dtype)
        choice = torch.stack([torch.randperm(5, generator=torch.Generator().manual_seed(t))[:2] for t in range(tokens)]).int()
        weight = torch.rand((tokens, 2), generator=torch.Generator().manual_seed(1))
        L.check(x, L.moe(x, choice.cuda(), weight.cuda()), choice, weight)


@pytest.mark.parametrize("quant", QUANTS, ids=["q8_0", "q4_0", "q4_K"])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("n,top,hidden,ffn", [
    (1, 1, 256, 256), (3, 1, 256, 8192), (4, 2, 2048, 1024), (16, 16, 256, 768), (5, 3, 1280, 2816), (2, 1, 4096, 256),
    (2, 2, 4864, 512), (1, 1, 512, 20480), (16, 16, 1792, 256)])
def test_one_routed_token(quant, dtype, n, top, hidden, ffn):
    """Fewer tiles than CTAs, a few more, rows of 1 to 160 stages; routed and with the same choice given."""
    L = Layer(quant, n, hidden, ffn, top, seed=ffn, max_tokens=1)
    x = rand(9, 1, hidden, dtype=dtype)
    y, choice, weight = L.moe(x, routing=True)
    assert sorted(choice[0].tolist()) == sorted(set(choice[0].tolist())) and choice.max() < n
    L.check(x, y, choice, weight)
    L.check(x, L.moe(x, choice, weight), choice, weight)
    assert torch.equal(L.moe(x), y)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("rd", [F32, BF16], ids=["f32", "bf16"])
def test_routers(score, renormalize, biased, rd):
    bias = rand(4, 40) if biased else None
    L = Layer(O.Q4_0, 40, 128, 64, 6, router_dtype=rd, score=score, renormalize=renormalize, scale=2.5, bias=bias,
              act="gelu_tanh")
    x = rand(5, 21, 128, dtype=BF16)
    y, choice, weight = L.moe(x, routing=True)
    c, w, gap = P.route(x.cpu(), L.router.cpu(), bias.cpu() if biased else None, score, 6, renormalize, 2.5)
    assert gap > 1e-6
    assert torch.equal(choice.cpu(), c) and (weight.cpu().double() - w).abs().max() < 2.0 ** -17
    L.check(x, y, c, w)


def test_equal_scores_take_the_lowest_index_and_nan_is_the_least():
    L = Layer(O.Q4_0, 70, 64, 64, 5)
    L.router.zero_()
    x = rand(1, 3, 64)
    _, choice, weight = L.moe(x, routing=True)
    assert choice.tolist() == [[0, 1, 2, 3, 4]] * 3 and torch.allclose(weight, torch.full_like(weight, 0.2))
    L.router[[0, 2, 33]] = math.nan                      # their scores, for any token
    L.router[40, 0] = math.inf
    x[:, 0] = 1.0
    assert L.moe(x, routing=True)[1].tolist() == [[40, 1, 3, 4, 5]] * 3


def test_choices_of_the_caller():
    """No expert, an index out of range, an expert twice, a token with none at all."""
    L = Layer(O.Q4_K, 6, 256, 256, 4, router=False, max_tokens=8)
    x = rand(2, 5, 256)
    choice = torch.tensor([[0, -1, 5, 6], [3, 3, 3, 3], [-1, -1, -7, 1 << 30], [5, 4, 5, 0], [1, 0, 2, -(1 << 31)]], dtype=torch.int32)
    weight = torch.rand((5, 4), generator=torch.Generator().manual_seed(3)) - 0.3
    weight[2] = math.nan                                 # of no expert: not looked at
    y = L.moe(x, choice.cuda(), weight.cuda())
    assert (y[2] == 0).all()
    L.check(x, y, choice, weight)
    assert (L.moe(x, torch.full_like(choice, -1).cuda(), weight.cuda()) == 0).all()


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_every_token_to_the_same_expert(dtype):
    """128 tokens of one expert are 16 passes over its weights; the others have none."""
    L = Layer(O.Q8_0, 9, 128, 96, 1, router=False, max_tokens=128)
    for tokens in (8, 9, 127, 128):
        x = rand(tokens, tokens, 128, dtype=dtype)
        choice, weight = torch.full((tokens, 1), 8, dtype=torch.int32), torch.rand((tokens, 1)) + 0.5
        L.check(x, L.moe(x, choice.cuda(), weight.cuda()), choice, weight)


def test_one_token_sixteen_times_to_one_expert_of_512():
    L = Layer(O.Q4_0, 512, 64, 64, 16, router=False, max_tokens=128)
    x = rand(1, 128, 64, dtype=BF16)
    choice = torch.full((128, 16), 511, dtype=torch.int32)          # 2048 pairs, 256 units of one expert
    weight = torch.full((128, 16), 1 / 16)
    L.check(x, L.moe(x, choice.cuda(), weight.cuda()), choice, weight)


@pytest.mark.parametrize("quant", QUANTS, ids=["q8_0", "q4_0", "q4_K"])
@pytest.mark.parametrize("dtype,sizes", [(F32, (1e-12, 1e-3, 1.0, 1e5, 3e12)), (BF16, (1e-12, 1e-3, 1.0, 1e5, 3e12))],
                         ids=["f32", "bf16"])
def test_tokens_of_any_size_beside_one_another(quant, dtype, sizes):
    """relu goes with the square of x, as the scales of the kernels do; a zero token; one channel far above the rest."""
    L = Layer(quant, 4, 256, 256, 2, router=False, act="relu")
    x = rand(5, len(sizes) + 2, 256, dtype=F32)
    for i, s in enumerate(sizes):
        x[i] *= s
    x[-2] = 0
    x[-1, 77] = 4e4
    x = x.to(dtype)
    choice = torch.tensor([[i % 4, (i + 1) % 4] for i in range(len(x))], dtype=torch.int32)
    weight = torch.full((len(x), 2), 0.5)
    y = L.moe(x, choice.cuda(), weight.cuda())
    assert (y[-2] == 0).all()
    L.check(x, y, choice, weight)


def test_a_token_that_is_not_finite_touches_no_other():
    L = Layer(O.Q4_0, 4, 256, 128, 2)
    x = rand(6, 12, 256, dtype=BF16)
    want = L.moe(x)
    bad = x.clone()
    bad[3, 5], bad[7, 0] = math.nan, math.inf
    got = L.moe(bad)
    keep = [i for i in range(12) if i not in (3, 7)]
    # the others' experts and places may share passes with other tokens, but not their numbers
    L.check(x[keep], got[keep], *L.moe(x[keep], routing=True)[1:])
    assert not torch.isfinite(got[3]).any() and torch.equal(L.moe(x), want)


def test_strided_tokens_and_what_is_behind_them():
    L = Layer(O.Q8_0, 4, 64, 64, 2, max_tokens=16)
    wide = rand(7, 11, 160, dtype=BF16)
    x = wide[:, 32:96]
    out = torch.full((14, 80), 9.0, device="cuda", dtype=BF16)
    y = L.moe(x, out=out[:11, :64])
    assert torch.equal(y, L.moe(x.contiguous()))
    assert (out[11:] == 9).all() and (out[:, 64:] == 9).all()
    L.moe(x, out=x)                                      # over its own input: read before it is written
    assert torch.equal(x, y)
    assert L.moe(x[:0]).shape == (0, 64)
    L.check(wide[:1, 96:], L.moe(wide[:1, 96:]), *L.moe(wide[:1, 96:], routing=True)[1:])


def test_graphs_that_share_a_workspace_and_other_streams():
    L = Layer(O.Q4_0, 32, 256, 128, 4, max_tokens=64)
    a, b = rand(1, 50, 256, dtype=BF16), rand(2, 1, 256, dtype=F32)
    wa, wb = L.moe(a), L.moe(b)
    ga, gb = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(ga):
        oa = L.moe(a)
    with torch.cuda.graph(gb):
        ob = L.moe(b)
    for _ in range(5):                                   # in turn, on one stream
        ga.replay()
        gb.replay()
    torch.cuda.synchronize()
    assert torch.equal(oa, wa) and torch.equal(ob, wb)
    a.copy_(rand(9, 50, 256))
    ga.replay()
    assert torch.equal(oa, L.moe(a))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out = L.moe(b)
    side.synchronize()
    assert torch.equal(out, wb)


def test_two_layers_in_one_stream():
    """Calls one behind the other, each with a workspace of its own, chained without a wait between them."""
    A, C = Layer(O.Q4_0, 16, 256, 128, 4, seed=3), Layer(O.Q8_0, 8, 256, 64, 2, seed=4)
    x = rand(1, 33, 256, dtype=BF16)
    one = A.moe(x)
    torch.cuda.synchronize()
    two = C.moe(one)
    torch.cuda.synchronize()
    for _ in range(10):
        got = C.moe(A.moe(x))
    assert torch.equal(got, two)


def test_experts_of_a_loaded_base():
    from quantized_base_lora_gb300.runtime import Runtime
    rng = np.random.default_rng(2)
    n, hidden, ffn = 4, 256, 512
    shapes = [(n * ffn, hidden), (n * ffn, hidden), (n * hidden, ffn)]
    for quant in QUANTS:
        base = S.build_base(quant, [(0, i, S.gaussian(rng, s, 0.05)) for i, s in enumerate(shapes)])
        rt = Runtime(arena_bytes=32 << 20)
        tensors = [(t.layer, t.proj, t.d_out, t.d_in, t.qs_off, t.d_off) for t in base.tensors]
        q.check(rt.load_base(base.quant, tensors, base.buf, S.content_digest(base.buf)), rt.ctx)
        w = []
        for (qs, d), (rows, cols) in zip(base.planes, shapes):
            w.append(torch.from_numpy(np.asarray(O.dequantize(quant, qs, d), np.float64)).reshape(n, -1, cols))
        router = rand(3, n, hidden, scale=0.2)
        moe = B.Moe.from_base(rt, 0, 1, 2, n, 2, router=router)
        x = rand(4, 6, hidden, dtype=BF16)
        y, choice, weight = moe(x, routing=True)
        L = Layer.__new__(Layer)
        L.w, L.act = w, "silu"
        L.check(x, y, choice.cpu(), weight.cpu())
        with pytest.raises(ValueError):
            B.Moe.from_base(rt, 0, 2, 1, n, 2, router=router)
        rt.close()


def test_what_the_torch_side_refuses():
    L = Layer(O.Q4_0, 4, 64, 64, 2, max_tokens=4)
    x = rand(1, 3, 64)
    c, w = torch.zeros((3, 2), dtype=torch.int32, device="cuda"), torch.zeros((3, 2), device="cuda")
    for call in (lambda: L.moe(rand(1, 5, 64)), lambda: L.moe(x.half()), lambda: L.moe(x[:, :32]), lambda: L.moe(x.cpu()),
                 lambda: L.moe(x, c), lambda: L.moe(x, weight=w), lambda: L.moe(x, c.long(), w), lambda: L.moe(x, c, w.double()),
                 lambda: L.moe(x, c[:2], w), lambda: L.moe(x, c, w[:, :1]), lambda: L.moe(x, c, w, routing=True),
                 lambda: L.moe(x, out=x[:2]), lambda: L.moe(x, out=x.bfloat16())):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(q.OvlError):
        Layer(O.Q4_0, 4, 64, 64, 2, router=False).moe(x)
    planes = L.moe._held[:3]
    for n, kw in ((4, dict(router=rand(1, 4, 32))), (4, dict(bias=rand(1, 5))), (3, {}), (4, dict(score="top")), (4, dict(act="no"))):
        with pytest.raises(ValueError):
            B.Moe(O.Q4_0, n, 64, 64, *planes, top_k=2, **kw)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("tokens", [1, 3, 11])
def test_activations_keep_their_bits_between_the_products(dtype, tokens):
    """Outputs that are the difference of two activations, of up to 19 bits each: what is cut off them shows in full.

    x is one channel, so that g = 1 and u = 127 d x come out of their products exactly but for a rounding or two, and a
    down row has the codes 127 and -127 (the 7 bits that an MMA holds).  Three parts are all 24 bits of an activation;
    six MMAs cut their sums at 2^-23 of the larger product and a handful of steps round by 2^-24: below 2^-20 of both."""
    rng = np.random.default_rng(tokens)
    hidden, ffn = 256, 256
    gate, up = np.zeros((ffn, hidden), np.int8), np.zeros((ffn, hidden), np.int8)
    gate[:, 0], up[:, 0] = 64, 127
    gd = np.full((ffn, hidden // 32), 1 / 64, np.float16)
    ud = np.broadcast_to((1 + rng.integers(0, 1024, (ffn, 1)) / 1024).astype(np.float16), gd.shape)
    down, one, two = np.zeros((hidden, ffn), np.int8), np.arange(hidden), (np.arange(hidden) + rng.integers(1, ffn, hidden)) % ffn
    down[one, one], down[one, two] = 127, -127
    dd = np.full((hidden, ffn // 32), 1 / 128, np.float16)
    planes = [tuple(torch.from_numpy(np.ascontiguousarray(p)).cuda() for p in pl) for pl in ((gate, gd), (up, ud), (down, dd))]
    moe = B.Moe(O.Q8_0, 1, hidden, ffn, *planes, top_k=1, act="relu")
    x = torch.zeros((tokens, hidden))
    x[:, 0] = 1 + torch.arange(tokens) / 128                 # bf16 values
    y = moe(x.to(dtype).cuda(), torch.zeros((tokens, 1), dtype=torch.int32, device="cuda"), torch.ones((tokens, 1), device="cuda"))
    h = x[:, :1].double() ** 2 * 127 * torch.from_numpy(ud[:, 0].astype(np.float64))
    a, b = h[:, one] * 127 / 128, h[:, two] * 127 / 128
    off = (y.double().cpu() - (a - b)).abs()
    assert (off <= 2.0 ** -20 * (a + b) + P.HALF[dtype] * (a - b).abs() * 1.001).all(), float((off / (a + b)).max() * 2 ** 20)


def test_a_workspace_that_calls_raced_on_is_right_again_for_the_next():
    """Counters as overlapping calls leave them, and choices of no expert: the next call clears the counters, whatever
    it answers itself (here no CTA finds itself the last, so nothing is chosen), and the one after it is as ever."""
    L = Layer(O.Q4_0, 40, 128, 64, 3, max_tokens=16)         # five router CTAs of 8 experts for each 8 tokens
    words = L.moe.workspace.view(torch.int32)
    choice = 64 + 16 * 40                                    # behind the counters and the logits
    for tokens in (11, 1):
        x, other = rand(tokens, tokens, 128, dtype=BF16), rand(9, tokens, 128, dtype=BF16)
        want = L.moe(other, routing=True)
        assert torch.equal(words[choice:choice + 3 * tokens].view(tokens, 3), want[1])
        words[:16] = 1000
        words[choice:choice + 3 * tokens] = torch.tensor([-5, 40, 1 << 30], dtype=torch.int32, device="cuda").repeat(tokens)
        L.moe(x)
        assert (words[:16] == 0).all()
        for a, b in zip(L.moe(other, routing=True), want):
            assert torch.equal(a, b)


def test_experts_under_an_active_overlay_are_refused():
    """Low-rank and sparse, in a stack and in a table; on another tensor, taken back or rolled back they do not matter."""
    from quantized_base_lora_gb300.runtime import Runtime
    rng = np.random.default_rng(5)
    shapes = [(64, 32), (64, 32), (64, 32), (64, 32)]        # two experts of 32 x 32, and another projection
    base = S.build_base(S.Q8_0, [(0, i, S.gaussian(rng, s, 0.05)) for i, s in enumerate(shapes)])
    rt = Runtime(arena_bytes=32 << 20)
    assert q.ovl_count_overlays(rt.ctx, [0]) == (q.OVL_E_STATE, 0)
    q.check(rt.load_base(base.quant, [(t.layer, t.proj, t.d_out, t.d_in, t.qs_off, t.d_off) for t in base.tensors], base.buf,
                         S.content_digest(base.buf)), rt.ctx)

    def lora(*tensors):
        ad = S.build_adapter(base, list(tensors), [4] * len(tensors),
                             [(S.gaussian(rng, (4, 32), 0.1), S.gaussian(rng, (64, 4), 0.1)) for _ in tensors])
        st, h = rt.stage(ad, S.content_digest(ad.payload))
        q.check(st, rt.ctx)
        return h

    def sparse(tensor):
        sp = S.build_sparse_adapter([tensor], [S.dare_entries(rng, 64, 32, 0.1)])
        st, h = rt.stage_sparse(sp, S.content_digest(sp.payload))
        q.check(st, rt.ctx)
        return h

    moe = B.Moe.from_base(rt, 0, 1, -2, 2, 1, router=rand(1, 2, 32))
    x = rand(2, 3, 32)
    want = moe(x)
    other, two, one = lora(3), lora(3, 2), sparse(0)
    for handles, mode, count in (([other], q.OVL_MODE_STACK, 0), ([other, two], q.OVL_MODE_STACK, 1), ([two], q.OVL_MODE_TABLE, 1),
                                 ([one, other, two], q.OVL_MODE_STACK, 2), ([], q.OVL_MODE_STACK, 0)):
        q.check(rt.activate(handles, [1.0] * len(handles), mode)[0], rt.ctx)
        assert q.ovl_count_overlays(rt.ctx, [0, 1, 2]) == (0, count)
        if count:
            for call in (lambda: moe(x), lambda: B.Moe.from_base(rt, 0, 1, 2, 2, 1)):
                with pytest.raises(q.OvlError) as e:
                    call()
                assert e.value.status == q.OVL_E_STATE
        else:
            assert torch.equal(moe(x), want)
    assert q.ovl_count_overlays(rt.ctx, [3, 4])[0] == q.OVL_E_ARG and q.ovl_count_overlays(rt.ctx, []) == (0, 0)
    q.check(rt.rollback()[0], rt.ctx)
    with pytest.raises(q.OvlError):
        moe(x)
    rt.close()
    assert torch.equal(moe(x), want)                     # the base's planes are kept


@pytest.mark.parametrize("score,bias,logits", [
    ("sigmoid", None, [-100.0, -95.5, -110.25, -98.125, -103.0, -95.625]),       # all below what fp32 scores hold
    ("sigmoid", None, [-89.0, -90.0, -89.5, -91.0, -300.0, -89.125]),
    ("sigmoid", None, [3.0, -100.0, -0.5, 0.0, 12.0, -20.0]),
    ("sigmoid", [0, 5, 4, 0, 3, 0], [2.0, -120.0, -130.0, 1.0, -121.5, 0.0]),    # far-off ones by their bias
    ("softmax", [0, 5, 4, 0, 3, 0], [2.0, -120.0, -130.0, 1.0, -121.5, 0.0]),
    ("softmax", [0, 5, 4, 0, 3, 0], [88.0, -20.0, -18.0, 1.0, -15.5, 0.0]),      # subnormal ones
    ("softmax", None, [500.0, 499.0, -500.0, 498.5, 0.0, 480.0])])
@pytest.mark.parametrize("top", [1, 3])
def test_weights_of_scores_that_32_bits_do_not_hold(score, bias, logits, top):
    """Divided by their sum, weights go by the scores' ratios, however small the scores are.

    x is a unit, so logits are exact, and so are their differences: e^ to 2 ulp, a sum and a quotient, 2^-20 in all."""
    n = len(logits)
    b = None if bias is None else torch.tensor(bias, dtype=F32).cuda()
    x, router = torch.zeros((2, 64)), torch.zeros((n, 64))
    x[:, 0], router[:, 0] = 1.0, torch.tensor(logits)
    for renormalize in (True, False):
        L = Layer(O.Q4_0, n, 64, 64, top, score=score, bias=b, renormalize=renormalize, scale=0.5)
        L.router.copy_(router)
        y, choice, weight = L.moe(x.cuda(), routing=True)
        c, w, _ = P.route(x, router, None if b is None else b.cpu(), score, top, renormalize, 0.5)
        assert torch.equal(choice.cpu(), c)
        assert ((weight.cpu().double() - w).abs() <= 2.0 ** -20 * w + 2.0 ** -148).all(), (weight, w)
        if renormalize:                                  # else weights of 2^-140 make outputs whose steps are 2^-149
            L.check(x.cuda(), y, c, w)

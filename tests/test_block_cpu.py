"""The operators between a block's projections without a device: the rotation's plan, the statements that the GPU
tests compare with, and what the library and its torch side refuse before they touch a device."""
import ctypes
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import block_plain as P  # noqa: E402
import oracle as O  # noqa: E402


@pytest.fixture(scope="module")
def q():
    return pytest.importorskip("quantized_base_lora_gb300")


# ---------------------------------------------------------------- the rotation's plan

@pytest.mark.parametrize("scaling,kind", [(None, 0), ("linear", 1), ("base", 2), ("bands", 3), ("ramp", 4)])
@pytest.mark.parametrize("dim,rot,base,factor,original", [(128, 128, 500000.0, 8.0, 8192), (96, 40, 10000.0, 2.5, 4096),
                                                         (64, 2, 10000.0, 4.0, 512), (512, 510, 1e6, 32.0, 32768)])
def test_plan_against_the_formula(q, scaling, kind, dim, rot, base, factor, original):
    low, high = {"bands": (1.0, 4.0), "ramp": (1.0, 32.0)}.get(scaling, (1.0, 4.0))
    st, plan = q.ovl_rope_plan(dim, rot, q.OVL_ROPE_HALF, base, kind, factor, original, low, high)
    assert st == 0 and (plan.head_dim, plan.rot_dim) == (dim, rot)
    w, size = P.frequencies(rot, base, scaling, factor, original)
    got = np.array(list(plan.turn)[:rot // 2], np.float64) * math.tau / 2.0 ** 64
    # both sides: a power of up to 40 ulp and a handful of roundings of 2^-53; the fixed point's step, 2^-64 of a turn,
    # is cut off: 2 pi 2^-64 = 3.5e-19 radians at most
    np.testing.assert_allclose(got, w, rtol=2.0 ** -46, atol=math.tau * 2.0 ** -64)
    assert plan.magnitude == np.float32(size) and all(t == 0 for t in list(plan.turn)[rot // 2:])


def test_plan_by_hand(q):
    _, plan = q.ovl_rope_plan(4, 4, q.OVL_ROPE_PAIRS, 100.0, magnitude=2.5)
    assert plan.turn[0] / 2.0 ** 64 == pytest.approx(1 / math.tau) and plan.magnitude == 2.5
    assert plan.turn[1] / 2.0 ** 64 == pytest.approx(0.1 / math.tau)
    # the wrap-around of the product is the reduction by whole turns
    pos = 123456789
    phase = (pos * plan.turn[0]) % 2 ** 64 / 2.0 ** 64 * math.tau
    assert math.sin(phase) == pytest.approx(math.sin(pos), abs=1e-7)


@pytest.mark.parametrize("args,status", [
    ((0, 0, 1, 1e4), "SHAPE"), ((7, 4, 1, 1e4), "SHAPE"), ((514, 4, 1, 1e4), "SHAPE"), ((64, 3, 1, 1e4), "SHAPE"),
    ((64, 66, 1, 1e4), "SHAPE"), ((64, 0, 1, 1e4), "SHAPE"), ((64, 64, 3, 1e4), "ARG"), ((64, 64, 1, 1.0), "ARG"),
    ((64, 64, 1, math.nan), "ARG"), ((64, 64, 1, math.inf), "ARG"), ((64, 64, 1, 1e4, 5), "ARG"),
    ((64, 64, 1, 1e4, 1, 0.5), "ARG"), ((64, 64, 1, 1e4, 1, math.inf), "ARG"), ((64, 64, 1, 1e4, 3, 2.0, 0), "ARG"),
    ((64, 64, 1, 1e4, 3, 2.0, 8, 4.0, 4.0), "ARG"), ((64, 64, 1, 1e4, 4, 2.0, 8, 0.0, 4.0), "ARG"),
    ((64, 64, 1, 1e4, 0, 1.0, 0, 1.0, 4.0, -1.0), "ARG"), ((64, 64, 1, 1e300, 2, 1e300), "ARG"),
])
def test_plans_that_are_refused(q, args, status):
    assert q.ovl_rope_plan(*args)[0] == getattr(q, f"OVL_E_{status}")
    assert q.ovl_last_error(None)


# ---------------------------------------------------------------- the statements

def test_rotation_by_hand():
    x = torch.tensor([[[1.0, 0.0, 5.0, 7.0]]], dtype=torch.float64)
    pos = torch.tensor([1])
    y, mag = P.rope(x, pos, [math.pi / 2], 1.0, "pairs")
    np.testing.assert_allclose(y[0, 0], [0, 1, 5, 7], atol=1e-15)
    np.testing.assert_allclose(mag[0, 0], [1, 1, 0, 0])
    y, _ = P.rope(x, pos, [math.pi / 2, 0.0], 2.0, "half")
    np.testing.assert_allclose(y[0, 0], [-10, 0, 2, 14], atol=1e-14)


def test_norms_by_hand():
    v = torch.tensor([[3.0, -1.0]], dtype=torch.float64)
    np.testing.assert_allclose(P.normed(v, "rms", None, None, 0.0, 0.0)[0][0], [3 / 5 ** 0.5, -1 / 5 ** 0.5])
    w, b = torch.tensor([1.0, 3.0]), torch.tensor([10.0, 20.0])
    np.testing.assert_allclose(P.normed(v, "layer", w, b, 0.0, 1.0)[0][0], [12, 16])


@pytest.mark.parametrize("quant", [O.Q8_0, O.Q4_0, O.Q4_K])
def test_experts_are_the_bases_formats(quant):
    (qs, d), w = P.experts(np.random.default_rng(1), quant, 2, 3, 256)
    one = O.dequantize(quant, qs[3:4], d[3:4] if quant == O.Q4_K else d[3:4].view(np.uint16))
    np.testing.assert_array_equal(w[1, 0].numpy(), np.asarray(one, np.float64)[0])
    assert 0.3 < w.std() * 16 < 3


def test_experts_add_up_by_hand():
    one = torch.ones((2, 1, 1), dtype=torch.float64)
    x = torch.tensor([[2.0]], dtype=torch.float64)
    y, _ = P.moe(x, one, 3 * one, one, torch.tensor([[1, 1, -1, 7]]), torch.tensor([[0.5, 0.25, 9.0, 9.0]]), "relu", True)
    assert y.item() == 0.75 * 2 * 6


def test_route_takes_the_lowest_index_of_equals():
    x, r = torch.ones((1, 4)), torch.zeros((6, 4))
    choice, w, gap = P.route(x, r, None, "softmax", 3, False, 2.0)
    assert choice.tolist() == [[0, 1, 2]] and gap == 0
    np.testing.assert_allclose(w, 2 / 6)


# ---------------------------------------------------------------- refusals: the library

AT = 1 << 20      # an address that no call gets as far as to use


def rope_call(q, plan=None, **kw):
    a = dict(n=4, pos=AT, qp=AT, qh=2, qs=16, k=AT, kh=1, ks=8, dt=1, qo=2 * AT, qos=16, ko=2 * AT, kos=8, odt=1)
    a.update(kw)
    plan = plan or q.ovl_rope_plan(8, 8, 1, 1e4)[1]
    return q.ovl_rope_apply(plan, a["n"], a["pos"], a["qp"], a["qh"], a["qs"], a["k"], a["kh"], a["ks"], a["dt"], a["qo"],
                            a["qos"], a["ko"], a["kos"], a["odt"])


@pytest.mark.parametrize("kw,status", [
    (dict(pos=0), "ARG"), (dict(pos=AT + 2), "SHAPE"), (dict(qp=0), "ARG"), (dict(k=0), "ARG"), (dict(qo=0), "ARG"),
    (dict(ko=0), "ARG"), (dict(dt=3), "ARG"), (dict(odt=0), "ARG"), (dict(qh=0), "SHAPE"), (dict(qh=65536), "SHAPE"),
    (dict(kh=65536), "SHAPE"), (dict(qs=15), "SHAPE"), (dict(ks=7), "SHAPE"), (dict(qos=15), "SHAPE"),
    (dict(kos=0), "SHAPE"), (dict(qp=AT + 2), "SHAPE"), (dict(n=1 << 31), "ARG"), (dict(qs=(1 << 31) + 1), "SHAPE"),
    (dict(qo=AT, qos=32), "SHAPE"), (dict(qo=AT, odt=2), "SHAPE"), (dict(ko=AT, kos=16), "SHAPE"),
])
def test_rotations_that_are_refused(q, kw, status):
    assert rope_call(q, **kw) == getattr(q, f"OVL_E_{status}")


def test_a_rotation_that_no_plan_made_is_refused(q):
    assert rope_call(q, q.ovl_rope()) == q.OVL_E_SHAPE
    assert q.lib.ovl_rope_apply(None, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0) == q.OVL_E_ARG
    assert rope_call(q, n=0, pos=0, qp=0) == 0


def norm_call(q, pre=1, post=0, hidden=8, eps=1e-6, offset=0.0, alpha=1.0, beta=1.0, w=None, w_dtype=1, **kw):
    a = dict(n=4, x=AT, xd=1, xs=8, y=AT, yd=1, ys=8, g=0, gd=1, gs=8, gr=0, ng=0, xo=AT, xos=8, h=2 * AT, hd=1, hs=8)
    a.update(kw)
    plan = q.ovl_block_norm(hidden, alpha, beta, q.ovl_norm(post, w_dtype, w, None, eps, offset),
                            q.ovl_norm(pre, w_dtype, w, None, eps, offset))
    return q.ovl_block_norm_apply(plan, a["n"], a["x"], a["xd"], a["xs"], a["y"], a["yd"], a["ys"], a["g"], a["gd"],
                                  a["gs"], a["gr"], a["ng"], a["xo"], a["xos"], a["h"], a["hd"], a["hs"])


@pytest.mark.parametrize("kw,status", [
    (dict(hidden=0), "SHAPE"), (dict(hidden=32769), "SHAPE"), (dict(pre=3), "ARG"), (dict(post=3), "ARG"),
    (dict(eps=-1.0), "ARG"), (dict(eps=math.nan), "ARG"), (dict(offset=math.inf), "ARG"), (dict(alpha=math.nan), "ARG"),
    (dict(beta=math.inf), "ARG"), (dict(w=AT, w_dtype=0), "ARG"), (dict(w=AT + 1), "SHAPE"), (dict(x=0), "ARG"),
    (dict(xd=3), "ARG"), (dict(yd=0), "ARG"), (dict(hd=7), "ARG"), (dict(xs=7), "SHAPE"), (dict(ys=7), "SHAPE"),
    (dict(hs=7), "SHAPE"), (dict(xos=9), "SHAPE"), (dict(x=AT + 1), "SHAPE"), (dict(h=0), "ARG"),
    (dict(pre=0), "ARG"), (dict(pre=0, h=0, xo=0), "ARG"), (dict(g=AT), "ARG"), (dict(g=AT, ng=3), "SHAPE"),
    (dict(g=AT, ng=4, gs=7), "SHAPE"), (dict(g=AT, ng=4, gd=0), "ARG"), (dict(g=AT, ng=4, gr=AT + 1), "SHAPE"),
    (dict(n=1 << 31), "ARG"),
])
def test_norms_that_are_refused(q, kw, status):
    assert norm_call(q, **kw) == getattr(q, f"OVL_E_{status}")


@pytest.mark.parametrize("args,status", [
    ((0, 4, 8, AT, 8, AT, 8, 1, AT, 8, 1), "ARG"), ((5, 4, 8, AT, 8, AT, 8, 1, AT, 8, 1), "ARG"),
    ((1, 4, 0, AT, 8, AT, 8, 1, AT, 8, 1), "SHAPE"), ((1, 4, 8, 0, 8, AT, 8, 1, AT, 8, 1), "ARG"),
    ((1, 4, 8, AT, 7, AT, 8, 1, AT, 8, 1), "SHAPE"), ((1, 4, 8, AT, 8, AT, 7, 1, AT, 8, 1), "SHAPE"),
    ((1, 4, 8, AT, 8, AT, 8, 1, AT, 9, 1), "SHAPE"), ((1, 4, 8, AT, 8, AT, 8, 1, AT, 8, 2), "SHAPE"),
    ((1, 4, 8, AT, 8, AT, 8, 3, AT, 8, 1), "ARG"), ((1, 1 << 31, 8, AT, 8, AT, 8, 1, AT, 8, 1), "ARG"),
    ((1, 4, 8, AT, 8, AT + 2, 8, 1, AT, 8, 1), "SHAPE"),
])
def test_activations_that_are_refused(q, args, status):
    assert q.ovl_glu(*args) == getattr(q, f"OVL_E_{status}")


def layer(q, **kw):
    a = dict(quant=2, n_experts=8, top_k=2, hidden=64, ffn=96, act=1, score=1, renormalize=1, scale=1.0, router_dtype=1,
             max_tokens=16, gate_qs=AT, gate_d=AT, up_qs=AT, up_d=AT, down_qs=AT, down_d=AT, router=AT, bias=None,
             workspace=AT, workspace_bytes=1 << 30)
    a.update(kw)
    return q.ovl_moe(**a)


def moe_call(q, m, x=AT, dt=1, n=4, xs=64, choice=0, weight=0, co=0, wo=0, y=2 * AT, ys=64):
    return q.ovl_moe_forward(m, x, dt, n, xs, choice, weight, co, wo, y, ys)


@pytest.mark.parametrize("kw,status", [
    (dict(quant=0), "QUANT"), (dict(quant=4), "QUANT"), (dict(n_experts=0), "ARG"), (dict(n_experts=513), "ARG"),
    (dict(top_k=0), "ARG"), (dict(top_k=9), "ARG"), (dict(n_experts=64, top_k=17), "ARG"), (dict(hidden=0), "SHAPE"),
    (dict(hidden=48), "SHAPE"), (dict(ffn=100), "SHAPE"), (dict(quant=3), "SHAPE"), (dict(hidden=32800), "SHAPE"),
    (dict(act=0), "ARG"), (dict(act=5), "ARG"), (dict(max_tokens=0), "ARG"), (dict(max_tokens=129), "ARG"),
])
def test_layers_that_are_refused(q, kw, status):
    m = layer(q, **kw)
    assert q.ovl_moe_workspace_bytes(m) == (getattr(q, f"OVL_E_{status}"), 0)
    assert moe_call(q, m) == getattr(q, f"OVL_E_{status}")


@pytest.mark.parametrize("kw,call,status", [
    (dict(gate_qs=None), {}, "ARG"), (dict(down_d=None), {}, "ARG"), (dict(workspace=None), {}, "ARG"),
    (dict(up_qs=AT + 8), {}, "SHAPE"), (dict(workspace=AT + 16), {}, "SHAPE"), (dict(workspace_bytes=1000), {}, "OOM"),
    (dict(router=None), {}, "ARG"), (dict(router=AT + 4), {}, "SHAPE"), (dict(bias=AT + 2), {}, "SHAPE"),
    (dict(score=0), {}, "ARG"), (dict(score=3), {}, "ARG"), (dict(router_dtype=0), {}, "ARG"),
    (dict(scale=math.nan), {}, "ARG"), ({}, dict(choice=AT), "ARG"), ({}, dict(weight=AT), "ARG"),
    ({}, dict(choice=AT, weight=AT, co=AT), "ARG"), ({}, dict(choice=AT, weight=AT, wo=AT), "ARG"),
    ({}, dict(choice=AT + 2, weight=AT), "SHAPE"), ({}, dict(n=17), "ARG"), ({}, dict(dt=0), "ARG"),
    ({}, dict(x=0), "ARG"), ({}, dict(y=0), "ARG"), ({}, dict(xs=63), "SHAPE"), ({}, dict(xs=66), "SHAPE"),
    ({}, dict(ys=65), "SHAPE"), ({}, dict(x=AT + 8), "SHAPE"), ({}, dict(dt=2, ys=68), "SHAPE"),
])
def test_calls_of_a_layer_that_are_refused(q, kw, call, status):
    assert moe_call(q, layer(q, **kw), **call) == getattr(q, f"OVL_E_{status}")


def test_a_call_without_tokens_is_nothing(q):
    assert moe_call(q, layer(q), n=0, x=0, y=0) == 0
    assert norm_call(q, n=0, x=0, y=0, h=AT) == 0
    assert q.ovl_glu(1, 0, 8, 0, 8, 0, 8, 1, 0, 8, 1) == 0


def test_workspace_grows_with_what_it_holds(q):
    st, size = q.ovl_moe_workspace_bytes(layer(q))
    # 16 tokens: 3 bf16 parts of 64, and of 96 for each of 2 experts, and 64 fp32 of each
    assert st == 0 and 16 * (6 * 64 + 2 * 6 * 96 + 2 * 4 * 64) <= size < 40000
    assert q.ovl_moe_workspace_bytes(layer(q, max_tokens=128))[1] > 7 * size


def test_positions_that_are_refused(q):
    kv = q.ovl_kv(AT, AT, AT, AT, AT, AT, 1 << 30, 8, 16, 1, 1, 64, 4, 4)
    for args, status in (((0, AT, 1, 4, AT), "ARG"), ((AT, AT, 1, 4, 0), "ARG"), ((AT, AT, 1, 4, AT + 2), "SHAPE"),
                         ((AT, AT, 1025, 4, AT), "ARG"), ((AT, AT, 1, 1 << 31, AT), "ARG")):
        assert q.ovl_kv_positions(kv, *args) == getattr(q, f"OVL_E_{status}")
    assert q.ovl_kv_positions(kv, AT, AT, 0, 4, AT) == 0


def test_packed_calls(q):
    import struct

    def call(which, *words):
        return q.ovl_packed(which, struct.pack(f"={len(words)}Q", *words), len(words))

    plan, norm, moe = q.ovl_rope_plan(8, 8, 1, 1e4)[1], q.ovl_block_norm(8, 1.0, 1.0), layer(q)
    norm.pre.kind = 1
    at = ctypes.addressof
    rope = [at(plan), 0, AT, AT, 2, 16, AT, 1, 8, 1, 2 * AT, 16, 2 * AT, 8, 1]
    block = [at(norm), 0, AT, 1, 8, AT, 1, 8, 0, 1, 0, 0, 0, AT, 8, 2 * AT, 1, 8]
    glu = [1, 0, 8, AT, 8, AT, 8, 1, AT, 8, 1]
    experts = [at(moe), AT, 1, 0, 64, 0, 0, 0, 0, 2 * AT, 64]
    calls = [(q.OVL_PACKED_ROPE, rope), (q.OVL_PACKED_BLOCK_NORM, block), (q.OVL_PACKED_GLU, glu), (q.OVL_PACKED_MOE, experts)]
    for which, words in calls:
        assert call(which, *words) == 0                  # no tokens: checked, and nothing to do
        assert call(which, *words, 0) == q.OVL_E_ARG and call(which, *words[:-1]) == q.OVL_E_ARG
    # every argument is in its place: what each refuses is refused
    for which, words, i, v, status in (
            (1, rope, 0, 0, "ARG"), (1, rope, 4, 0, "SHAPE"), (1, rope, 7, 70000, "SHAPE"), (1, rope, 9, 5, "ARG"),
            (1, rope, 14, 0, "ARG"), (1, rope, 1, 1 << 32, "ARG"), (2, block, 0, 0, "ARG"), (2, block, 3, 0, "ARG"),
            (2, block, 6, 9, "ARG"), (2, block, 15, 0, "ARG"), (2, block, 16, 4, "ARG"), (2, block, 9, 1 << 40, "ARG"),
            (3, glu, 0, 7, "ARG"), (3, glu, 2, 0, "SHAPE"), (3, glu, 7, 0, "ARG"), (3, glu, 10, 3, "ARG"),
            (4, experts, 0, 0, "ARG"), (4, experts, 2, 0, "ARG"), (4, experts, 3, 17, "ARG"), (4, experts, 5, AT, "ARG"),
            (4, experts, 3, 1 << 32, "ARG")):
        assert call(which, *(words[:i] + [v] + words[i + 1:])) == getattr(q, f"OVL_E_{status}"), (which, i)
    # and where there are tokens, of the tensors
    for which, words, n, bad in ((1, rope, 1, (2, 3, 6, 10, 12)), (2, block, 1, (2,)), (3, glu, 1, (3, 5, 8)), (4, experts, 3, (1, 9))):
        some = words[:n] + [4] + words[n + 1:]
        for i in bad:
            assert call(which, *(some[:i] + [0] + some[i + 1:])) == q.OVL_E_ARG, (which, i)
    for which, words, n, strides in ((1, rope, 1, (5, 8, 11, 13)), (2, block, 1, (4, 7, 14, 17)), (3, glu, 1, (4, 6, 9)),
                                     (4, experts, 3, (4, 10))):
        some = words[:n] + [4] + words[n + 1:]
        for i in strides:
            assert call(which, *(some[:i] + [1] + some[i + 1:])) == q.OVL_E_SHAPE, (which, i)
    assert call(0) == call(5, *glu) == q.OVL_E_ARG and q.lib.ovl_packed(1, None, 15, None) == q.OVL_E_ARG


def test_constants_match_the_header(q):
    import os
    import re
    with open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "ovl.h")) as f:
        text = f.read()
    found = re.findall(r"\b(OVL_(?:ROPE|NORM|ACT|MOE|PACKED)_[A-Z_0-9]+) = (\d+)", text)
    assert len(found) >= 20
    for name, value in found:
        assert getattr(q, name) == int(value), name


# ---------------------------------------------------------------- refusals: the torch side

def test_torch_side_refuses_what_is_not_on_a_device(q):
    from quantized_base_lora_gb300 import block as B
    x = torch.zeros((2, 64))
    with pytest.raises(ValueError):
        B.Rope(64)(torch.zeros(2, dtype=torch.int32), x.view(2, 1, 64))
    with pytest.raises(ValueError):
        B.BlockNorm(64, B.Norm("rms"))(x)
    with pytest.raises(ValueError):
        B.BlockNorm(64, B.Norm("rms", torch.ones(64)))
    with pytest.raises(ValueError):
        B.glu(x, x)
    for make in (lambda: B.Rope(64, layout="other"), lambda: B.Rope(64, scaling="other"),
                 lambda: B.BlockNorm(64, B.Norm("other")), lambda: B.Rope(-2), lambda: B.BlockNorm(-1, None),
                 lambda: B.Moe(2, -1, 64, 64, None, None, None, 2)):
        with pytest.raises(ValueError):
            make()
    with pytest.raises(q.OvlError):
        B.Rope(63)
    assert ctypes.sizeof(q.ovl_rope) == 16 + 8 * 256


# ---------------------------------------------------------------- what the torch side keeps

def test_a_copied_or_pickled_rope_has_a_plan_of_its_own(q, monkeypatch):
    """The plan that a call hands to the library is the object's own, also after the one it was copied from is gone."""
    import copy
    import pickle
    import struct

    from quantized_base_lora_gb300 import block as B
    seen = []
    monkeypatch.setattr(B, "_call", lambda index, which, words: seen.append(struct.unpack("=15Q", words)[0]))
    monkeypatch.setattr(B, "_index_of", lambda name, t: t.get_device())
    monkeypatch.setattr(B, "_ints", lambda name, t, shape, index: t.data_ptr())
    pos, x = torch.zeros(2, dtype=torch.int32), torch.zeros((2, 1, 64))
    rope = B.Rope(64, 48, base=500000.0)
    want = bytes(rope.plan)
    for made in (rope, copy.copy(rope), copy.deepcopy(rope), pickle.loads(pickle.dumps(rope))):
        made(pos, x)
        assert seen.pop() == ctypes.addressof(made.plan) and bytes(made.plan) == want
    far = copy.deepcopy(rope)
    del rope, made
    far(pos, x)
    assert bytes((ctypes.c_char * len(want)).from_address(seen.pop())) == want


def test_weights_whose_storage_is_swapped_stay_alive(q, monkeypatch):
    """`parameter.data = other`, as Module.to does it, frees a storage that no one else holds: the addresses that the
    library reads have to be of tensors that the operator keeps."""
    from quantized_base_lora_gb300 import block as B
    monkeypatch.setattr(B, "_index_of", lambda name, t: t.get_device())

    def pointers(held):
        for h in held:
            yield from pointers(h) if isinstance(h, tuple) else () if h is None else (h.data_ptr(),)

    def swap(tensors):
        for t in tensors:
            t.data = torch.zeros_like(t)

    w = [torch.nn.Parameter(torch.ones(8)) for _ in range(4)]
    n = B.BlockNorm(8, B.Norm("rms", w[0], w[1]), B.Norm("layer", w[2], w[3]))
    swap(w)
    assert {n.plan.pre.weight, n.plan.pre.bias, n.plan.post.weight, n.plan.post.bias} <= set(pointers(n._held))
    assert all(torch.equal(t, torch.ones(8)) for t in n._held)
    planes = [(torch.zeros((64, 32), dtype=torch.int8), torch.zeros((64, 1), dtype=torch.float16)) for _ in range(3)]
    router, bias = torch.nn.Parameter(torch.ones((2, 32))), torch.nn.Parameter(torch.ones(2))
    m = B.Moe(q.OVL_Q8_0, 2, 32, 32, *planes, top_k=1, router=router, bias=bias)
    at = {getattr(m.moe, f) for f in ("gate_qs", "gate_d", "up_qs", "up_d", "down_qs", "down_d", "router", "bias")}
    swap([router, bias] + [t for pair in planes for t in pair])
    assert len(at) == 8 and at <= set(pointers(m._held))


@pytest.mark.parametrize("dim,base", [(128, 500000.0), (256, 1e6), (128, 10000.0), (512, 1e12)])
def test_plans_frequencies_are_rounded_to_the_nearest_step(q, dim, base):
    """2^-64 of a turn is the step: half of it, and 2^-46 of the frequency itself as above."""
    from fractions import Fraction
    _, plan = q.ovl_rope_plan(dim, dim, q.OVL_ROPE_HALF, base)
    tau = Fraction(6283185307179586476925286766559, 10 ** 30)
    for i, turn in enumerate(list(plan.turn)[:dim // 2]):
        w = Fraction(math.pow(base, -2 * i / dim))           # off by 2^-46 of itself at most
        want = w / tau * 2 ** 64
        assert abs(turn - want) <= Fraction(1, 2) + want * Fraction(1, 2 ** 46)


def test_positions_of_no_sequence_are_left_as_they_are(q):
    """No sequences are a no-op of the library, as in every call of the cache: pos is not written."""
    kv = q.ovl_kv(AT, AT, AT, AT, AT, AT, 1 << 30, 8, 16, 1, 1, 64, 4, 4)
    pos = (ctypes.c_int32 * 4)(7, 7, 7, 7)
    assert q.ovl_kv_positions(kv, 0, 0, 0, 4, ctypes.addressof(pos)) == 0 and list(pos) == [7] * 4

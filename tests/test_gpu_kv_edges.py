"""The 4-bit cache where calls, sizes or values are out of the ordinary."""
import numpy as np
import pytest

import kv_plain as K

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_kv import dev, draw, fill, make, offsets  # noqa: E402

if torch.cuda.is_available():
    import quantized_base_lora_gb300 as q


def latched(c, status):
    with pytest.raises(q.OvlError) as e:
        c.check()
    assert e.value.status == status
    c.check()


# ---------------------------------------------------------------- tokens that no sequence owns

@pytest.mark.parametrize("kv,bf16", [(1, False), (1, True), (64, True)], ids=["f32", "bf16", "many rows"])
@pytest.mark.parametrize("off,stray,served", [
    ([0, 30, 47], [(47, 60)], [(0, 0, 30), (1, 30, 47)]),            # a call padded to 60 tokens
    ([2, 30, 60], [(0, 2)], [(0, 2, 30), (1, 30, 60)]),
    ([0, 20, 99], [(20, 60)], [(0, 0, 20)]),                         # an offset beyond the tokens
    ([0, -1, 60], [(0, 60)], []),                                    # neither part can be used
    ([0, 60, 20], [], [(0, 0, 60)]),                                 # falls back: the second has no tokens
    ([0, 0, 0], [(0, 60)], []),
])
def test_tokens_of_no_sequence_are_zero_and_latched(kv, bf16, off, stray, served):
    rng = np.random.default_rng(sum(off) & 0xff)
    c = make(n_pages=20, page=16, kv=kv, dim=64, rows=4, cols=8)
    held = fill(c, [3, 1], [90, 70], rng, bf16=bf16)
    x = draw(rng, (60, 4 * kv, 64), bf16)
    wide = torch.full((60, 4 * kv + 1, 64), float("nan"), device="cuda", dtype=x.dtype)
    c.attention(0, dev([3, 1]), dev(off), x, 60, out=wide[:, 1:])
    latched(c, q.OVL_E_ARG)
    assert torch.isnan(wide[:, 0]).all()                             # nothing beside the rows
    got = wide[:, 1:].double().cpu().numpy()
    for a, b in stray:
        assert (got[a:b] == 0).all()
    for i, a, b in served:
        k, v = held[[3, 1][i]]
        w, spread, top = K.attention(x[a:b].double().cpu().numpy(), k, v,
                                     np.arange(k.shape[0] - (b - a), k.shape[0]), 0.125)
        assert (np.abs(got[a:b] - w) <= K.allowed(w, spread, top, bf16)).all()


def test_a_call_without_sequences_returns_zeros():
    c = make(kv=1, dim=64)
    none, off = dev([]), dev([0])
    x = torch.ones((5, 4, 64), device="cuda")
    for t in (c.attention(0, none, off, x, 1), c.attention(0, none, off, x, 1, out=torch.ones_like(x)),
              *c.read(0, none, off, 3)):
        assert (t == 0).all()
    c.check()

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


# ---------------------------------------------------------------- precision of bf16 calls

@pytest.mark.parametrize("dim,most", [(64, 1), (128, 1), (256, 1), (64, 9), (128, 9)])   # 9: two tiles of rows
def test_scores_of_bf16_calls_are_32_bit(dim, most):
    """Queries of one sign and two keys whose scores, in the thousands, all but agree: what the scores lose is what the
    outputs show.  A score is summed in 32 bits, three roundings a block of partial sums that are at most
    C = scale sum d code |q|, each within 2^-23 and most of them of a part of C: 2^-22 C in the mean square is more
    than that.  Two tokens of weight near 1/2 and values near +-1: half of the difference of their two errors.  The
    weights are rounded to 11 bits twice, the output to 8."""
    rng = np.random.default_rng(dim + most)
    n, kv, blocks = 64, 8, dim // 32
    qs = torch.from_numpy((8 * 2 ** (-6 * rng.random((n, kv, dim)))).astype(np.float32)).bfloat16()
    x = qs.double().numpy()
    a = rng.integers(4, 7, (n, kv, dim))
    a[..., ::32] = 8                                                 # the block's largest: d = 1 / 8
    b = a.copy()
    for i in range(n):
        for h in range(kv):
            u, w = rng.permutation(blocks)[:2]                       # two blocks; of 31 x 31 pairs the closest queries
            cu, cw = np.arange(32 * u + 1, 32 * u + 32), np.arange(32 * w + 1, 32 * w + 32)
            far = np.abs(x[i, h, cu][:, None] - x[i, h, cw][None])
            at = np.where(far > 0, far, 9).argmin()
            b[i, h, cu[at // 31]] -= 1
            b[i, h, cw[at % 31]] += 1
    k = torch.from_numpy(np.stack([a, b], 1).reshape(2 * n, kv, dim).astype(np.float32) / 8).cuda()
    v = torch.ones((2 * n, kv, dim), device="cuda")
    v[1::2] = -1
    c = make(n_pages=n, page=16, kv=kv, dim=dim, rows=n, cols=1)
    rows, off = dev(range(n)), dev(np.arange(n + 1) * 2)
    c.extend(rows, off)
    c.append(0, rows, off, k, v)
    scale = 4096 / dim
    got = c.attention(0, rows, dev(range(n + 1)), qs.cuda(), most, scale=scale).double().cpu().numpy()
    c.check()
    want, size = np.empty_like(got), 0.0
    kk, vv = (K.values_of(*K.quantize(t.cpu().numpy())).reshape(n, 2, kv, dim) for t in (k, v))
    for i in range(n):
        out, spread, _ = K.attention(x[i:i + 1], kk[i], vv[i], [1], scale)
        want[i], size = out[0], max(size, float((spread * (8 + 7) / 7).max()))        # code <= (8 + 7) / 7 |code - 8| here
    assert size > 8000 and np.abs(want).mean() < 0.25
    rms = np.sqrt(((got - want) ** 2).mean())
    assert rms <= 2 ** -22 * size * 2 ** 0.5 / 2 + 2 ** -11 + 2 ** -9 * np.sqrt((want ** 2).mean()), (rms, size)


@pytest.mark.parametrize("size", [1e-6, 1.0, 2e5])
@pytest.mark.parametrize("dim,most", [(64, 1), (128, 1), (256, 1), (64, 9), (128, 9)])
def test_a_tail_of_small_weights_at_any_size_of_values(dim, most, size):
    """Every 64th token far above the others, which hold 2 % of the weight together and all of the value but in channel
    0: whatever the values' size is, the weights of the others may not fall out of f16.  Scores are good to 2^-18 of
    sum |q k| (32-bit sums), weights rounded to 11 bits twice, the output to 8."""
    rng = np.random.default_rng(dim + most)
    n, kv = 6000, 32
    c = make(n_pages=n // 64 + 1, page=64, kv=kv, dim=dim, rows=1, cols=n // 64 + 1, garbage=False)
    k = torch.zeros((n, kv, dim), device="cuda")
    k[17::64, :, 0] = -8.0                                           # held exactly: code 0, d = 1
    v = draw(rng, (n, kv, dim)).abs().clamp(0.5, 2.0) * (size / 2)
    v[17::64] = 0
    v[17::64, :, 0] = -size
    rows, off = dev([0]), dev([0, n])
    c.extend(rows, off)
    c.append(0, rows, off, k, v)
    x = torch.zeros((1, kv, dim), device="cuda", dtype=torch.bfloat16)
    x[:, :, 0] = -1.5
    scale = 11.5 * np.log(2) / 12                                    # the others 2^-11.5 of such a token's weight
    got = c.attention(0, rows, dev([0, 1]), x, most, scale=scale).double().cpu().numpy()
    c.check()
    kk, vv = (K.values_of(*K.quantize(t.cpu().numpy())) for t in (k, v))
    w, spread, top = K.attention(x.double().cpu().numpy(), kk, vv, [n - 1], scale)
    assert (np.abs(got - w) <= (2 ** -17 * spread + 2 ** -10) * top + 2 ** -8 * np.abs(w)).all(), \
        float(np.abs(got - w).max() / size)


# ---------------------------------------------------------------- sizes

def test_more_row_tiles_than_the_grid_of_the_kernel_for_many_rows():
    """16.8 million rows of one sequence.  A window of one token: every row returns its own token's values."""
    rng = np.random.default_rng(0)
    n, group = 16400, 1024
    assert n * group > 65535 * 256
    c = make(n_pages=n // 256 + 1, page=256, kv=1, dim=64, rows=1, cols=n // 256 + 1, garbage=False)
    rows, off = dev([0]), dev([0, n])
    c.extend(rows, off)
    k, v = draw(rng, (n, 1, 64), True), draw(rng, (n, 1, 64), True)
    c.append(0, rows, off, k, v)
    x = torch.ones((n, group, 64), device="cuda", dtype=torch.bfloat16)
    out = c.attention(0, rows, off, x, n, window=1)
    c.check()
    want = c.read(0, rows, off, n)[1]
    for i in range(0, n, 1024):
        w = want[i:i + 1024]
        assert ((out[i:i + 1024].float() - w).abs() <= 2 ** -8 * w.abs()).all()


# ---------------------------------------------------------------- pages of more than one row

@pytest.mark.parametrize("kv,bf16", [(1, False), (2, True), (64, True)])       # 64: several heads a thread
def test_tokens_are_not_written_into_pages_that_another_row_holds(kv, bf16):
    """A fork between extend and append: the new tokens' full pages are shared by then."""
    rng = np.random.default_rng(kv)
    new = 100 if kv == 64 else 20                                    # tokens 40 ..: 40 .. 47 in the third page
    c = make(n_pages=20, page=16, kv=kv, dim=128, rows=3, cols=12)
    held = fill(c, [0], [40], rng, bf16=bf16)[0]
    row, off = dev([0]), dev([0, new])
    c.extend(row, off)
    c.fork(row, dev([1]))
    before = c.codes.clone(), c.scales.view(torch.int16).clone()
    k, v = draw(rng, (new, kv, 128), bf16), draw(rng, (new, kv, 128), bf16)
    c.append(0, row, off, k, v)
    latched(c, q.OVL_E_STATE)
    shared = c.refs > 1
    assert int(shared.sum()) == (40 + new) // 16
    assert torch.equal(c.codes[shared], before[0][shared])
    assert torch.equal(c.scales.view(torch.int16)[shared], before[1][shared])
    for got, x in zip(c.read(0, row, dev([0, (40 + new) % 16]), (40 + new) % 16), (k, v)):   # the open page is its own
        own = K.values_of(*K.quantize(x[new - (40 + new) % 16:].float().cpu().numpy()))
        np.testing.assert_array_equal(got.cpu().numpy(), own.astype(np.float32))
    c.release(dev([1]))
    c.append(0, row, off, k, v)
    c.check()
    for got, x, old in zip(c.read(0, row, dev([0, 40 + new]), 40 + new), (k, v), held):
        want = np.concatenate([old, K.values_of(*K.quantize(x.float().cpu().numpy()))])
        np.testing.assert_array_equal(got.cpu().numpy(), want.astype(np.float32))


@pytest.mark.parametrize("small", [2.0 ** -12, 2.0 ** -8])
@pytest.mark.parametrize("dim,kv,new", [(128, 1, 1), (64, 2, 4), (128, 40, 60), (64, 40, 60), (256, 40, 60)])
def test_blocks_of_very_different_size(dim, kv, new, small):
    """Within 2^-14 of a tile's largest scale every block of channels keeps its bits: small values beside large ones."""
    rng = np.random.default_rng(dim + new)
    n = 300
    c = make(n_pages=20, page=16, kv=kv, dim=dim, rows=1, cols=20)
    rows, off = dev([0]), dev([0, n])
    c.extend(rows, off)
    k, v = draw(rng, (n, kv, dim)), draw(rng, (n, kv, dim))
    k[..., :32] *= small
    v[..., 32:64] *= small
    k, v = k.bfloat16(), v.bfloat16()
    c.append(0, rows, off, k, v)
    c.check()
    x = draw(rng, (new, 8 * kv, dim), True)
    got = c.attention(0, rows, dev([0, new]), x, new).double().cpu().numpy()
    c.check()
    kk, vv = (K.values_of(*K.quantize(t.float().cpu().numpy())) for t in (k, v))
    w, spread, top = K.attention(x.double().cpu().numpy(), kk, vv, np.arange(n - new, n), dim ** -0.5)
    assert (np.abs(got - w) <= K.allowed(w, spread, top, True)).all()
    block = np.s_[..., 32:64]
    assert np.sqrt(((got - w)[block] ** 2).mean()) <= 2 ** -8 * np.sqrt((w[block] ** 2).mean())


# ---------------------------------------------------------------- kernels that overlap their launches

@pytest.mark.parametrize("kv,new", [(2, 1), (40, 30)], ids=["few rows", "many rows"])
def test_steps_without_a_pause_give_what_steps_with_pauses_give(kv, new):
    """Each kernel is resident while the one before still runs: pages, tokens and queries written just before."""
    def run(pause):
        g = torch.Generator("cuda").manual_seed(3)
        c = make(n_pages=160, page=16, layers=2, kv=kv, dim=128, rows=4, cols=60, garbage=False)
        c.scales.fill_(float("nan"))
        rows, off = dev([2, 0]), dev([0, new, 2 * new])
        outs = []
        for step in range(24):
            calls = [lambda: c.extend(rows, off)]
            for layer in range(2):
                k, v, x = (torch.randn((2 * new, h, 128), generator=g, device="cuda").bfloat16()
                           for h in (kv, kv, 4 * kv))
                calls += [lambda layer=layer, k=k, v=v: c.append(layer, rows, off, k, v),
                          lambda layer=layer, x=x: outs.append(c.attention(layer, rows, off, x, new))]
            calls += [lambda: c.fork(dev([2]), dev([1]))] if step % 5 == 4 else []
            for call in calls:
                call()
                if pause:
                    torch.cuda.synchronize()
        c.check()
        return torch.cat(outs)

    a, b = run(False), run(True)
    assert torch.isfinite(a).all() and torch.equal(a, b)


# ---------------------------------------------------------------- queries of any size

@pytest.mark.parametrize("size", [-118, 0, 119, 125, 127])
@pytest.mark.parametrize("kv,new,bf16", [(1, 1, False), (1, 1, True), (2, 4, True), (40, 60, True)],
                         ids=["f32", "bf16", "bf16-2", "many rows"])
def test_queries_of_any_size(size, kv, new, bf16):
    """Queries up to the type's end and down to where their scale makes up for it."""
    rng = np.random.default_rng(size & 0xff)
    c = make(n_pages=20, page=16, kv=kv, dim=64, rows=1, cols=20)
    held = fill(c, [0], [200], rng, bf16=bf16)
    x = draw(rng, (new, 8 * kv, 64), bf16).clamp(-1.9, 1.9) * 2.0 ** size
    assert torch.isfinite(x).all()
    x[:, 0, 0] = 1.9 * 2.0 ** size                                   # the size is reached in some row
    scale = max(0.125 * 2.0 ** -size, 2.0 ** -126)                   # a normal number
    got = c.attention(0, dev([0]), dev([0, new]), x, new, scale=scale).double().cpu().numpy()
    c.check()
    w, spread, top = K.attention(x.double().cpu().numpy(), *held[0], np.arange(200 - new, 200), scale)
    assert (np.abs(got - w) <= K.allowed(w, spread, top, bf16)).all()

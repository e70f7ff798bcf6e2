"""Attention over the 4-bit cache where many tokens are weighed: the error in the mean square against 64 bits, which
does not shrink into the worst case's bound as the context grows, and which kernel it is that is tested."""
import numpy as np
import pytest

import kv_plain as K

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_kv import dev, draw, fill, make, offsets  # noqa: E402

if torch.cuda.is_available():
    import quantized_base_lora_gb300 as q

FEW, SINGLE, PAIRS = range(3)

# A bf16 result is off by up to 2^-8 of itself, 1.6 to 1.7e-3 in the mean square; what else is rounded (weights twice to
# 11 bits; with many rows keys and values to 11 bits) is below 5e-4 where scores stay below 10.  f32: exp and sums of
# some thousand tokens, 2^-22 each.
RMS = {True: 2.0 ** -8, False: 2.0 ** -18}


def rms(x):
    return float(np.sqrt((np.asarray(x) ** 2).mean()))


def route(c, new, heads, bf16):
    st, r = q.ovl_debug_kv_route(c.kv, len(new), sum(new), max(new), q.OVL_BF16 if bf16 else q.OVL_F32, heads,
                                 torch.cuda.get_device_properties(0).multi_processor_count)
    assert st == q.OVL_OK
    return r


def judged(c, held, rows, new, group, rng, bf16, want_route, window=0, sinks=0, slices=()):
    """Attention of the rows' last tokens; each sequence's error in the mean square, and the worst case.  slices: tokens
    of the first row without which the 64-bit result would be far outside of the limit."""
    heads, dim = c.n_kv_heads * group, c.head_dim
    assert route(c, new, heads, bf16) == want_route
    off = offsets(new)
    x = draw(rng, (int(off[-1]), heads, dim), bf16)
    got = c.attention(0, dev(rows), dev(off), x, max(new), window=window, sinks=sinks)
    c.check()
    got, x = got.double().cpu().numpy(), x.double().cpu().numpy()
    for i, row in enumerate(rows):
        k, v = held.get(row, (np.zeros((0, c.n_kv_heads, dim)),) * 2)
        n, t = k.shape[0], new[i]
        if t == 0:
            continue
        a, b = off[i], off[i + 1]
        if n == 0:
            assert (got[a:b] == 0).all()
            continue
        pos = np.arange(n - t, n)
        want, spread, top = K.attention(x[a:b], k, v, pos, dim ** -0.5, window, sinks)
        assert (got[a:b][pos < 0] == 0).all()
        assert (np.abs(got[a:b] - want) <= K.allowed(want, spread, top, bf16)).all()
        limit = RMS[bf16] * rms(want)
        assert rms(got[a:b] - want) <= limit, (row, rms(got[a:b] - want) / rms(want))
        for at, size in slices if i == 0 else ():
            rest = np.r_[0:at, at + size:n]
            less = K.attention(x[a:b], k[rest], v[rest], pos - size, dim ** -0.5)[0]
            assert rms(less - want) > 4 * limit


# ---------------------------------------------------------------- few rows

@pytest.mark.parametrize("bf16", [False, True], ids=["f32", "bf16"])
@pytest.mark.parametrize("dim,kv,group,new", [(128, 1, 4, 1), (64, 2, 4, 1), (256, 1, 2, 1), (128, 2, 4, 5), (64, 1, 8, 3)])
def test_few_rows_over_a_long_context(dim, kv, group, new, bf16):
    """Hundreds of partial results are joined; a lost tile of 32 tokens anywhere would show."""
    rng = np.random.default_rng(dim + new)
    n = 20000 if kv == 1 else 12000
    c = make(n_pages=700, page=32, kv=kv, dim=dim, rows=3, cols=n // 32 + 1)
    held = fill(c, [0, 2], [n, 701], rng, bf16=bf16)
    judged(c, held, [0, 2], [new, new], group, rng, bf16, FEW, slices=[(0, 32), (n // 2 // 32 * 32, 32), (n - 64, 32)])


def test_a_window_over_a_long_context():
    rng = np.random.default_rng(1)
    for bf16 in (False, True):
        c = make(n_pages=700, page=32, kv=2, dim=128, rows=3, cols=320)
        held = fill(c, [0, 2], [9000, 5000], rng, bf16=bf16)
        judged(c, held, [0, 2], [1, 1], 4, rng, bf16, FEW, window=3000, sinks=70)


# ---------------------------------------------------------------- many rows

@pytest.mark.parametrize("dim,page,kv,group,seqs,new,n,kernel", [
    (128, 64, 8, 4, 1, 400, 6000, PAIRS),
    (128, 16, 8, 4, 20, 60, 1500, SINGLE),
    (64, 32, 8, 8, 1, 300, 5000, SINGLE),
    (256, 64, 8, 4, 1, 200, 3000, SINGLE),
    (128, 256, 4, 8, 2, 333, 4000, PAIRS)])
def test_many_rows_over_a_long_context(dim, page, kv, group, seqs, new, n, kernel):
    """A lost half of a K or V tile, or an eighth of P's columns, would show."""
    rng = np.random.default_rng(new)
    c = make(n_pages=seqs * (n // page + 1), page=page, kv=kv, dim=dim, rows=seqs, cols=n // page + 1)
    rows = list(range(seqs))
    held = fill(c, rows, [n - 7 * i for i in rows], rng, bf16=True)
    judged(c, held, rows, [new - i for i in rows], group, rng, True, kernel,
           slices=[(0, 16), (n // 2 // 128 * 128, 16), (n - new - 48, 16)])


@pytest.mark.parametrize("window,sinks", [(700, 0), (900, 33)])
@pytest.mark.parametrize("dim,kv,group,new,kernel", [(128, 8, 4, 400, PAIRS), (64, 8, 8, 300, SINGLE), (256, 8, 4, 200, SINGLE)])
def test_many_rows_with_a_window_over_a_long_context(dim, kv, group, new, kernel, window, sinks):
    rng = np.random.default_rng(window + dim)
    c = make(n_pages=80, page=64, kv=kv, dim=dim, rows=1, cols=80)
    held = fill(c, [0], [4500], rng, bf16=True)
    judged(c, held, [0], [new], group, rng, True, kernel, window=window, sinks=sinks)


@pytest.mark.parametrize("dim,group", [(64, 8), (128, 8), (256, 8)])
def test_many_rows_with_nothing_to_see(dim, group):
    """The kernel for many rows: rows at positions below zero, a free row with many new tokens and one with one."""
    rng = np.random.default_rng(dim)
    c = make(n_pages=20, page=16, kv=40, dim=dim, rows=4, cols=8)
    held = fill(c, [0, 1], [25, 70], rng, bf16=True)
    kernel = SINGLE
    judged(c, held, [0, 3, 1, 2], [32, 20, 32, 1], group, rng, True, kernel)
    judged(c, held, [0, 1], [26, 30], group, rng, True, kernel, window=9, sinks=2)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_short_sequences_beside_a_long_one(dim):
    """Sequences of one and of no new token in a call that the kernel for many rows serves."""
    rng = np.random.default_rng(dim)
    c = make(n_pages=80, page=16, kv=64, dim=dim, rows=5, cols=45)
    held = fill(c, [0, 1, 2, 4], [600, 1, 40, 333], rng, bf16=True)
    judged(c, held, [0, 1, 2, 4], [200, 1, 0, 12], 4, rng, True, PAIRS if dim == 128 else SINGLE)
    judged(c, held, [1, 0, 4, 2], [1, 150, 13, 40], 4, rng, True, PAIRS if dim == 128 else SINGLE, window=100, sinks=3)

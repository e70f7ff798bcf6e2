"""The 4-bit key/value cache on the GPU: bytes written, values read, attention
against 64 bits, rows and pages against lists, refusals."""
import numpy as np
import pytest

import kv_plain as K

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import quantized_base_lora_gb300 as q
    from quantized_base_lora_gb300.kvcache import KvCache


def dev(x, dt=torch.int32):
    return torch.tensor(np.asarray(x), dtype=dt, device="cuda")


def make(n_pages=40, page=16, layers=1, kv=2, dim=64, rows=8, cols=16, garbage=True):
    """An empty cache; what no token has written is NaN scales and 0xff codes."""
    c = KvCache.allocate(n_pages, page, layers, kv, dim, rows, cols)
    if garbage:
        c.codes.fill_(255)
        c.scales.fill_(float("nan"))
    return c


def offsets(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def draw(rng, shape, bf16=False):
    x = torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).cuda()
    return x.bfloat16() if bf16 else x


def fill(c, seqs, lengths, rng, layer=0, bf16=False):
    """Extend the rows and write all their tokens; returns the values that the cache then stands for (64 bits), by row."""
    s, off = dev(seqs), dev(offsets(lengths))
    c.extend(s, off)
    total = int(sum(lengths))
    shape = (total, c.n_kv_heads, c.head_dim)
    k, v = draw(rng, shape, bf16), draw(rng, shape, bf16)
    c.append(layer, s, off, k, v)
    c.check()
    out = {}
    for i, row in enumerate(seqs):
        a, b = offsets(lengths)[i:i + 2]
        out[row] = tuple(K.values_of(*K.quantize(x[a:b].float().cpu().numpy())) for x in (k, v))
    return out


# ---------------------------------------------------------------- writing and reading

@pytest.mark.parametrize("dim,page,kv", [(64, 16, 1), (128, 64, 3), (256, 32, 2)])
@pytest.mark.parametrize("bf16", [False, True])
def test_append_writes_the_documented_bytes(dim, page, kv, bf16):
    rng = np.random.default_rng(dim + page)
    c = make(n_pages=12, page=page, layers=3, kv=kv, dim=dim)
    counts = [page + 3, 1, 0, 2 * page]
    s, off = dev([3, 0, 5, 1]), dev(offsets(counts))
    c.extend(s, off)
    total = sum(counts)
    wide = draw(rng, (total, 2, kv, dim), bf16)                  # k and v interleaved: strides that are not the shape's
    wide[0, 0, 0, :32] = 0                                       # a block with no scale
    wide[1, 1, kv - 1, 5] = float("inf")
    wide[2, 0, 0, 7] = float("nan")
    wide[3, 1, 0, 40:] = 1e-7
    k, v = wide[:, 0], wide[:, 1]
    c.append(1, s, off, k, v)
    c.check()
    table = c.table.cpu().numpy()
    codes, scales = c.codes.cpu().numpy(), c.scales.cpu().numpy()
    assert (codes[:, [0, 2]] == 255).all() and np.isnan(scales[:, [0, 2]]).all()      # other layers untouched
    at, written = 0, np.zeros(codes.shape[0] * page, bool)
    for row, n in zip([3, 0, 5, 1], counts):
        for which, x in ((0, k), (1, v)):
            want_c, want_d = K.quantize(x[at:at + n].float().cpu().numpy())
            for h in range(kv):
                got_c = np.concatenate([K.unpack(codes[p, 1, which, h], page, dim, which)
                                        for p in table[row] if p >= 0] or [np.zeros((0, dim))])[:n]
                got_d = np.concatenate([scales[p, 1, which, h] for p in table[row] if p >= 0]
                                       or [np.zeros((0, dim // 32))])[:n]
                np.testing.assert_array_equal(got_c, want_c[:, h])
                np.testing.assert_array_equal(got_d, want_d[:, h])
        written[[p * page + i for j, p in enumerate(table[row]) if p >= 0 for i in range(page) if j * page + i < n]] = 1
        at += n
    stays = ~written.reshape(-1, page)
    assert np.isnan(scales[:, 1].transpose(0, 3, 1, 2, 4)[stays]).all()               # nothing but the tokens' slots


def test_append_of_one_token_leaves_its_neighbours():
    rng = np.random.default_rng(5)
    c = make(page=16, kv=2, dim=128)
    held = fill(c, [0, 2], [15, 8], rng)
    s, off = dev([2, 0]), dev([0, 1, 2])
    c.extend(s, off)
    k, v = draw(rng, (2, 2, 128)), draw(rng, (2, 2, 128))
    c.append(0, s, off, k, v)
    for row, i in ((2, 0), (0, 1)):
        n = held[row][0].shape[0]
        got = c.read(0, dev([row]), dev([0, n + 1]), n + 1)
        for g, x, old in zip(got, (k, v), held[row]):
            new = K.values_of(*K.quantize(x[i:i + 1].cpu().numpy()))
            np.testing.assert_array_equal(g.cpu().numpy(), np.concatenate([old, new]).astype(np.float32))
    c.check()


# ---------------------------------------------------------------- attention

def attend_and_compare(c, held, seqs, new, heads, rng, bf16, window=0, sinks=0, layer=0, scale=None, spike=0.0,
                       max_new=None):
    dim = c.head_dim
    off = offsets(new)
    total = int(off[-1])
    x = draw(rng, (total, heads, dim), bf16)
    if spike:
        x = x * spike
    got = c.attention(layer, dev(seqs), dev(off), x, max_new or max(max(new), 1), scale=scale, window=window,
                      sinks=sinks)
    c.check()
    assert got.dtype == x.dtype and got.shape == x.shape
    got = got.double().cpu().numpy()
    x64 = x.double().cpu().numpy()
    for i, row in enumerate(seqs):
        k, v = held[row]
        n, t = k.shape[0], new[i]
        out, spread, top = K.attention(x64[off[i]:off[i + 1]], k, v, np.arange(n - t, n),
                                       scale if scale is not None else dim ** -0.5, window, sinks)
        d = np.abs(got[off[i]:off[i + 1]] - out)
        lim = K.allowed(out, spread, top, bf16)
        assert (d <= lim).all(), (row, float((d / lim).max()))
    return got


SHAPES = [
    # dim, page, kv, group, lengths, new
    (128, 64, 2, 4, [1, 63, 64, 65, 200], [1, 1, 1, 1, 1]),
    (64, 16, 1, 8, [1, 2, 31, 33, 17], [1, 2, 1, 1, 1]),
    (256, 32, 2, 1, [40, 7, 129], [1, 1, 1]),
    (128, 128, 1, 7, [130, 5], [3, 5]),                          # 21 rows: more than one tile of rows
    (128, 16, 3, 5, [90, 300, 1], [4, 2, 0]),                    # a sequence with no new token
    (64, 64, 2, 3, [97, 33], [33, 20]),
    (128, 32, 2, 4, [150, 40], [37, 40]),
    (256, 64, 1, 2, [140], [70]),
    (128, 256, 1, 1, [600], [1]),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"d{s[0]}p{s[1]}h{s[2]}x{s[3]}n{max(s[5])}")
@pytest.mark.parametrize("bf16", [False, True], ids=["f32", "bf16"])
def test_attention_against_64_bits(shape, bf16):
    dim, page, kv, group, lengths, new = shape
    rng = np.random.default_rng(sum(lengths) + dim)
    c = make(n_pages=60, page=page, kv=kv, dim=dim, rows=6, cols=-(-max(lengths) // page) + 1)
    rows = [4, 0, 2, 5, 1][:len(lengths)]
    held = fill(c, rows, lengths, rng, bf16=bf16)
    attend_and_compare(c, held, rows, new, kv * group, rng, bf16)


@pytest.mark.parametrize("window,sinks", [(1, 0), (5, 0), (16, 4), (33, 1), (40, 70), (1000, 4), (20, 17)])
@pytest.mark.parametrize("new", [1, 3, 50])
@pytest.mark.parametrize("bf16", [False, True], ids=["f32", "bf16"])
def test_window_and_sinks(window, sinks, new, bf16):
    rng = np.random.default_rng(window * 100 + sinks + new)
    c = make(n_pages=60, page=16, kv=2, dim=128, rows=4, cols=20)
    lengths = [250, new, 97]
    held = fill(c, [1, 0, 3], lengths, rng, bf16=bf16)
    attend_and_compare(c, held, [1, 0, 3], [new] * 3, 8, rng, bf16, window, sinks)


@pytest.mark.parametrize("new", [1, 60])
@pytest.mark.parametrize("bf16", [False, True], ids=["f32", "bf16"])
def test_sharp_and_flat_scores(new, bf16):
    """Scores that single one token out, scores that are all equal, and a negative scale."""
    rng = np.random.default_rng(new)
    kv = 48 if new > 1 else 1                                    # wide enough for the kernel for many rows
    c = make(n_pages=60, page=32, kv=kv, dim=128, rows=2, cols=16)
    held = fill(c, [0], [300], rng, bf16=bf16)
    for scale, spike in ((3.0, 4.0), (0.0, 1.0), (-0.2, 1.0)):
        attend_and_compare(c, held, [0], [new], 4 * kv, rng, bf16, scale=scale, spike=spike)


@pytest.mark.parametrize("new", [1, 60])
@pytest.mark.parametrize("size", [1e-6, 3e4])
def test_values_and_keys_of_any_size(new, size):
    """Scales at both ends of binary16: tiny and large keys and values, one token far above the others."""
    rng = np.random.default_rng(3)
    kv = 48 if new > 1 else 1                                    # wide enough for the kernel for many rows
    c = make(n_pages=20, page=32, kv=kv, dim=128, rows=2, cols=16)
    s, off, n = dev([0]), dev([0, 200]), 200
    c.extend(s, off)
    k, v = (draw(rng, (n, kv, 128), True).float() * size for _ in range(2))
    v[100] *= 3
    k, v = k.bfloat16(), v.bfloat16()
    c.append(0, s, off, k, v)
    held = {0: tuple(K.values_of(*K.quantize(x.float().cpu().numpy())) for x in (k, v))}
    attend_and_compare(c, held, [0], [new], 4 * kv, rng, True, scale=0.1 / size)


def test_long_context_split_over_many_blocks():
    rng = np.random.default_rng(9)
    for bf16 in (False, True):
        c = make(n_pages=400, page=64, kv=1, dim=128, rows=3, cols=330)
        held = fill(c, [0, 2], [20000, 700], rng, bf16=bf16)
        first = attend_and_compare(c, held, [0, 2], [1, 1], 4, np.random.default_rng(1), bf16)
        again = attend_and_compare(c, held, [0, 2], [1, 1], 4, np.random.default_rng(1), bf16)
        np.testing.assert_array_equal(first, again)              # the same inputs, the same bits


# Enough rows in all (new tokens x query heads / 16 x kv heads above four an SM) that bf16 calls go to the
# kernel for many rows.
WIDE = [
    # dim, page, kv, group, lengths, new
    (128, 64, 48, 2, [250, 97, 60], [50, 50, 33]),
    (64, 16, 40, 3, [300, 64, 33], [64, 64, 33]),
    (256, 32, 40, 1, [140, 129], [129, 70]),
    (128, 128, 64, 1, [600, 1, 40], [200, 1, 0]),                # and sequences of one token and of none
    (128, 16, 40, 7, [90, 45], [37, 45]),
    (64, 256, 48, 8, [513], [31]),
    (256, 16, 48, 2, [300, 20], [131, 3]),
]


@pytest.mark.parametrize("shape", WIDE, ids=lambda s: f"d{s[0]}p{s[1]}h{s[2]}x{s[3]}n{max(s[5])}")
@pytest.mark.parametrize("window,sinks", [(0, 0), (33, 1), (16, 70), (1000, 4), (1, 0)])
def test_many_rows(shape, window, sinks):
    dim, page, kv, group, lengths, new = shape
    rng = np.random.default_rng(sum(lengths) + window)
    c = make(n_pages=70, page=page, kv=kv, dim=dim, rows=5, cols=-(-max(lengths) // page) + 1)
    rows = [4, 0, 2][:len(lengths)]
    held = fill(c, rows, lengths, rng, bf16=True)
    attend_and_compare(c, held, rows, new, kv * group, rng, True, window, sinks)


@pytest.mark.parametrize("dim,page,kv,group,new,window,sinks", [
    (128, 64, 16, 4, 300, 0, 0),       # 1200 rows: five tiles of rows, twelve tiles of tokens
    (128, 16, 32, 3, 97, 0, 0),
    (64, 32, 8, 8, 200, 300, 5),
    (256, 128, 20, 1, 260, 0, 0),
    (256, 16, 20, 2, 150, 200, 40),
    (128, 64, 24, 2, 230, 600, 300)])
def test_chunks_over_a_long_context(dim, page, kv, group, new, window, sinks):
    rng = np.random.default_rng(new)
    lengths = [1500, new, 700]
    c = make(n_pages=250, page=page, kv=kv, dim=dim, rows=3, cols=1500 // page + 1)
    held = fill(c, [2, 0, 1], lengths, rng, bf16=True)
    first = attend_and_compare(c, held, [2, 0, 1], [new, new, 3], kv * group, np.random.default_rng(1), True, window,
                               sinks)          # 3 new tokens in the same call: served beside the others
    again = attend_and_compare(c, held, [2, 0, 1], [new, new, 3], kv * group, np.random.default_rng(1), True, window,
                               sinks)
    np.testing.assert_array_equal(first, again)


# Sequences that end anywhere in the tiles of rows of their CTAs: so many rows that pairs of CTAs take them, and
# the longest just above one CTA's rows, where single CTAs do.
@pytest.mark.parametrize("new", [[130, 65, 100, 70], [65, 33, 33, 40]], ids=["pairs", "single"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (90, 3)])
def test_ragged_row_tiles(new, window, sinks):
    rng = np.random.default_rng(sum(new) + window)
    c = make(n_pages=40, page=64, kv=24, dim=128, rows=4, cols=7)
    lengths = [390, 65, 257, 128]
    held = fill(c, [2, 0, 3, 1], lengths, rng, bf16=True)
    attend_and_compare(c, held, [2, 0, 3, 1], new, 96, rng, True, window, sinks)


@pytest.mark.parametrize("bf16", [False, True], ids=["f32", "bf16"])
def test_many_sequences_of_every_length(bf16):
    rng = np.random.default_rng(11)
    lengths = list(range(1, 98, 3))
    c = make(n_pages=200, page=16, kv=2, dim=64, rows=len(lengths), cols=8)
    rows = list(rng.permutation(len(lengths)))
    held = fill(c, rows, lengths, rng, bf16=bf16)
    attend_and_compare(c, held, rows, [1] * len(rows), 6, rng, bf16)
    attend_and_compare(c, held, rows, [1 + i % 3 if n > 3 else 1 for i, n in enumerate(lengths)], 6, rng, bf16)


@pytest.mark.parametrize("bf16", [False, True], ids=["f32", "bf16"])
@pytest.mark.parametrize("new,kv", [(1, 1), (24, 1), (30, 64)])   # the last: the kernel for many rows
def test_tokens_with_nothing_to_see_are_zero(bf16, new, kv):
    """More new tokens than the row has: positions below zero see nothing."""
    rng = np.random.default_rng(2)
    c = make(page=16, kv=kv, dim=128)
    first = 5 if kv == 1 else 25
    held = fill(c, [0, 1], [first, 30], rng, bf16=bf16)
    extra = 3
    off = offsets([first + extra, new, 1])
    x = draw(rng, (int(off[-1]), 4 * kv, 128), bf16)
    out = torch.full_like(x, float("nan"))
    c.attention(0, dev([0, 1, 2]), dev(off), x, max(first + extra, new), out=out)   # row 2 is free: its token sees nothing
    got = out.double().cpu().numpy()
    assert (got[:extra] == 0).all() and (got[-1] == 0).all()
    for row, a, b in ((0, extra, off[1]), (1, off[1], off[2])):
        k, v = held[row]
        w, spread, top = K.attention(x[a:b].double().cpu().numpy(), k, v, np.arange(k.shape[0] - (b - a), k.shape[0]),
                                     128 ** -0.5)
        assert (np.abs(got[a:b] - w) <= K.allowed(w, spread, top, bf16)).all()
    c.check()


def test_strided_queries_outputs_and_another_stream():
    rng = np.random.default_rng(4)
    c = make(page=32, layers=2, kv=40, dim=64)
    held = fill(c, [3, 1], [50, 33], rng, layer=1, bf16=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for new, bf16 in (([1, 1], False), ([20, 9], False), ([50, 33], True)):   # the last: many rows
            off = offsets(new)
            wide = draw(rng, (int(off[-1]), 168, 64), bf16)
            x, out = wide[:, 4:164], torch.full((int(off[-1]), 163, 64), 7.0, device="cuda", dtype=wide.dtype)
            c.attention(1, dev([3, 1]), dev(off), x, max(new), out=out[:, 2:162])
            c.check()
            o = out.double().cpu().numpy()
            assert (o[:, :2] == 7).all() and (o[:, 162:] == 7).all()
            for i, row in enumerate([3, 1]):
                k, v = held[row]
                n = k.shape[0]
                w, spread, top = K.attention(x[off[i]:off[i + 1]].double().cpu().numpy(), k, v,
                                             np.arange(n - new[i], n), 0.125)
                assert (np.abs(o[off[i]:off[i + 1], 2:162] - w) <= K.allowed(w, spread, top, bf16)).all()


def test_pages_beyond_4_gib():
    """Pages at the far end of a pool of more than 2^32 bytes of codes."""
    rng = np.random.default_rng(6)
    c = make(n_pages=2200, page=64, layers=32, kv=8, dim=128, rows=3, cols=4, garbage=False)
    assert c.codes.numel() > 1 << 32
    c.refs[:2190] = 1
    held = fill(c, [0], [150], rng, layer=31, bf16=True)
    assert int(c.table[0, 0]) == 2190
    attend_and_compare(c, held, [0], [1], 32, rng, True, layer=31)
    attend_and_compare(c, held, [0], [150], 72, rng, True, layer=31)      # 1350 rows: the kernel for many
    c.fork(dev([0]), dev([1]))
    c.compact(dev([0]), dev([2]), dev(np.arange(0, 150, 3)), dev([0, 50]))
    c.check()
    for row, at in ((1, np.arange(150)), (2, np.arange(0, 150, 3))):
        for g, w in zip(c.read(31, dev([row]), dev([0, len(at)]), len(at)), held[0]):
            np.testing.assert_array_equal(g.cpu().numpy(), w[at].astype(np.float32))


def test_a_step_in_a_graph():
    """extend, append and attention captured once and replayed: the lengths live on the device."""
    rng = np.random.default_rng(8)
    c = make(n_pages=30, page=16, kv=1, dim=128, rows=2, cols=8, garbage=False)
    fill(c, [0, 1], [14, 30], rng, bf16=True)
    s, off = dev([0, 1]), dev([0, 1, 2])
    k, v, x = (torch.zeros((2, h, 128), device="cuda", dtype=torch.bfloat16) for h in (1, 1, 4))
    out = torch.zeros_like(x)

    def step():
        c.extend(s, off)
        c.append(0, s, off, k, v)
        c.attention(0, s, off, x, 1, out=out)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c.attention(0, s, off, x, 1, out=out)                    # once before the capture
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(4):
        for t in (k, v, x):
            t.copy_(draw(rng, tuple(t.shape), True))
        g.replay()
        for j, row in enumerate((0, 1)):
            n = 14 + 16 * row + i + 1
            kk, vv = (t.double().cpu().numpy() for t in c.read(0, dev([row]), dev([0, n]), n))
            w, spread, top = K.attention(x[j:j + 1].double().cpu().numpy(), kk, vv, [n - 1], 128 ** -0.5)
            assert (np.abs(out[j:j + 1].double().cpu().numpy() - w) <= K.allowed(w, spread, top, True)).all()
    c.check()


# ---------------------------------------------------------------- rows and pages

def same_rows(c, m):
    np.testing.assert_array_equal(c.table.cpu().numpy(), m.table())
    np.testing.assert_array_equal(c.length.cpu().numpy(), m.length)
    np.testing.assert_array_equal(c.refs.cpu().numpy(), m.refs)


@pytest.mark.parametrize("seed", range(6))
def test_rows_and_pages_against_lists(seed):
    """A random course of calls; after each, tables, lengths and counts, and what every row's tokens hold."""
    rng = np.random.default_rng(100 + seed)
    page = [16, 32][seed % 2]
    dim = [64, 128, 256][seed % 3]
    c = make(n_pages=int(rng.integers(20, 60)), page=page, layers=2, kv=2, dim=dim, rows=9, cols=7)
    m = K.Rows(c.refs.shape[0], page, 9, 7)
    text = [[np.zeros((0, 2, 2, dim)) for _ in range(2)] for _ in range(9)]       # [row][layer]: tokens, K|V, heads
    refused = 0
    for step in range(40):
        what = rng.choice(["extend", "extend", "fork", "compact", "release"])
        n = int(rng.integers(1, 5))
        dst = [int(x) for x in rng.permutation(9)[:n]]
        others = [r for r in range(9) if r not in dst]
        src = [d if rng.random() < 0.3 else int(rng.choice(others)) for d in dst]
        if rng.random() < 0.1:
            dst[-1] = dst[0]                                      # listed twice, unless there is but one
        err = None
        try:
            if what == "extend":
                more = [int(x) for x in rng.integers(0, 3 * page, n)]
                m.extend(dst, more)
            elif what == "fork":
                keep = [int(rng.integers(0, m.length[s] + 1)) if rng.random() < 0.6 else m.length[s] for s in src]
                whole = all(k == m.length[s] for k, s in zip(keep, src))
                m.fork(src, dst, keep)
            elif what == "compact":
                pick = [np.sort(rng.permutation(m.length[s])[:int(rng.integers(0, m.length[s] + 1))]) for s in src]
                m.compact(src, dst, [len(p) for p in pick])
            else:
                m.release(dst)
        except (MemoryError, KeyError) as e:
            err = e
        if what == "extend":
            off = offsets(more)
            c.extend(dev(dst), dev(off))
            if err is None and off[-1]:
                shape = (int(off[-1]), 2, dim)
                for layer in range(2):
                    kv = [draw(rng, shape) for _ in range(2)]
                    c.append(layer, dev(dst), dev(off), *kv)
                    val = np.stack([K.values_of(*K.quantize(x.cpu().numpy())) for x in kv], 1)
                    for i, d in enumerate(dst):
                        text[d][layer] = np.concatenate([text[d][layer], val[off[i]:off[i + 1]]])
        elif what == "fork":
            c.fork(dev(src), dev(dst), None if whole else dev(keep))
            if err is None:
                new = [[text[s][layer][:k] for layer in range(2)] for s, k in zip(src, keep)]
                for d, t in zip(dst, new):
                    text[d] = t
        elif what == "compact":
            c.compact(dev(src), dev(dst), dev(np.concatenate(pick)), dev(offsets([len(p) for p in pick])))
            if err is None:
                new = [[text[s][layer][p] for layer in range(2)] for s, p in zip(src, pick)]
                for d, t in zip(dst, new):
                    text[d] = t
        else:
            c.release(dev(dst))
            if err is None:
                for d in dst:
                    text[d] = [np.zeros((0, 2, 2, dim)) for _ in range(2)]
        if err is not None:
            refused += 1
            with pytest.raises(q.OvlError) as got:
                c.check()
            assert got.value.status == (q.OVL_E_OOM if isinstance(err, MemoryError) else q.OVL_E_DUPLICATE)
        c.check()
        same_rows(c, m)
        for layer in range(2):
            off = offsets(m.length)
            k, v = c.read(layer, dev(range(9)), dev(off), int(off[-1]))
            want = np.concatenate([text[r][layer] for r in range(9)])
            np.testing.assert_array_equal(k.cpu().numpy(), want[:, 0].astype(np.float32))
            np.testing.assert_array_equal(v.cpu().numpy(), want[:, 1].astype(np.float32))
    c.check()


def test_many_entries_and_pages():
    """More pages than one pass of the free-page scan, and hundreds of entries."""
    c = make(n_pages=9000, page=16, kv=1, dim=64, rows=1000, cols=6, garbage=False)
    m = K.Rows(9000, 16, 1000, 6)
    rng = np.random.default_rng(0)
    rows = [int(r) for r in rng.permutation(1000)[:500]]
    more = [int(x) for x in rng.integers(0, 97, 500)]
    c.extend(dev(rows), dev(offsets(more)))
    m.extend(rows, more)
    same_rows(c, m)
    free = [r for r in range(1000) if r not in set(rows)]
    c.fork(dev(rows), dev(free))
    m.fork(rows, free)
    same_rows(c, m)
    c.release(dev(rows))
    m.release(rows)
    same_rows(c, m)
    c.check()


def test_device_side_refusals_change_nothing():
    rng = np.random.default_rng(1)
    c = make(n_pages=6, page=16, kv=1, dim=64, rows=4, cols=3)
    fill(c, [0, 1], [20, 17], rng)
    before = [t.clone() for t in (c.table, c.length, c.refs, c.codes, c.scales.view(torch.int16))]

    def refused(status, call, *args):
        call(*args)
        with pytest.raises(q.OvlError) as e:
            c.check()
        assert e.value.status == status
        c.check()                                                # reported once
        for a, b in zip(before, (c.table, c.length, c.refs, c.codes, c.scales.view(torch.int16))):
            assert torch.equal(a, b)

    refused(q.OVL_E_OOM, c.extend, dev([2]), dev([0, 48]))       # 3 pages, 2 are free
    refused(q.OVL_E_OOM, c.extend, dev([0]), dev([0, 30]))       # 4 columns
    refused(q.OVL_E_ARG, c.extend, dev([4]), dev([0, 1]))
    refused(q.OVL_E_ARG, c.extend, dev([-1]), dev([0, 1]))
    refused(q.OVL_E_ARG, c.extend, dev([2]), dev([0, -3]))
    refused(q.OVL_E_DUPLICATE, c.extend, dev([2, 2]), dev([0, 1, 2]))
    refused(q.OVL_E_DUPLICATE, c.release, dev([1, 1]))
    refused(q.OVL_E_ARG, c.release, dev([7]))
    refused(q.OVL_E_ARG, c.fork, dev([0]), dev([2]), dev([21]))
    refused(q.OVL_E_DUPLICATE, c.fork, dev([0, 1]), dev([1, 2]))
    refused(q.OVL_E_ARG, c.compact, dev([0]), dev([2]), dev([0, 20]), dev([0, 2]))
    refused(q.OVL_E_ARG, c.compact, dev([0]), dev([2]), dev([0, -1]), dev([0, 2]))
    refused(q.OVL_E_ARG, c.compact, dev([0]), dev([2]), dev([0, 1]), dev([0, 3]))
    refused(q.OVL_E_ARG, c.compact, dev([0]), dev([2]), dev([0, 1]), dev([1, 2]))
    refused(q.OVL_E_OOM, c.compact, dev([0]), dev([2]), dev(np.arange(33) % 20), dev([0, 33]))


def test_tokens_out_of_reach_are_latched_and_the_rest_is_served():
    rng = np.random.default_rng(1)
    c = make(n_pages=6, page=16, kv=1, dim=64, rows=4, cols=3)
    held = fill(c, [0], [20], rng)
    k = draw(rng, (2, 1, 64))
    c.append(0, dev([9, 0]), dev([0, 1, 2]), k, k)
    with pytest.raises(q.OvlError) as e:
        c.check()
    assert e.value.status == q.OVL_E_ARG
    want = K.values_of(*K.quantize(k[1:].cpu().numpy())).astype(np.float32)
    got, _ = c.read(0, dev([0]), dev([0, 1]), 1)
    np.testing.assert_array_equal(got.cpu().numpy(), want)
    x = draw(rng, (2, 1, 64))
    for new in (1, 2):                                           # 2: more than max_new says
        off = dev([0, 1, 2]) if new == 1 else dev([0, 2])
        seqs = dev([-5, 0]) if new == 1 else dev([0])
        c.attention(0, seqs, off, x, 1)
        with pytest.raises(q.OvlError) as e:
            c.check()
        assert e.value.status == (q.OVL_E_ARG if new == 1 else q.OVL_E_SHAPE)
    got = c.attention(0, dev([-5, 0]), dev([0, 1, 2]), x, 1)
    assert (got[0] == 0).all() and (got[1] != 0).any()
    with pytest.raises(q.OvlError):
        c.check()
    wide = make(n_pages=20, page=16, kv=64, dim=64, rows=4, cols=3)
    held = fill(wide, [0], [40], rng, bf16=True)
    x2 = draw(rng, (60, 256, 64), True)
    got = wide.attention(0, dev([0, -1]), dev([0, 40, 60]), x2, 30)        # one row too long for max_new, one unknown
    with pytest.raises(q.OvlError):
        wide.check()
    k2, v2 = held[0]
    w, spread, top = K.attention(x2[:30].double().cpu().numpy(), k2, v2, np.arange(30), 0.125)
    assert (np.abs(got[:30].double().cpu().numpy() - w) <= K.allowed(w, spread, top, True)).all()
    assert (got[30:] == 0).all()
    wide.table[0, 1] = -7                                        # a page that is not there: rows that do not need it
    got = wide.attention(0, dev([0]), dev([0, 40]), x2[:40], 40).double().cpu().numpy()
    with pytest.raises(q.OvlError):
        wide.check()
    assert np.isfinite(got).all()
    w, spread, top = K.attention(x2[:16].double().cpu().numpy(), k2, v2, np.arange(16), 0.125)
    assert (np.abs(got[:16] - w) <= K.allowed(w, spread, top, True)).all()
    c.length[1] = 40                                             # a row that counts tokens but has no pages
    got = c.attention(0, dev([1]), dev([0, 1]), x[:1], 1)
    with pytest.raises(q.OvlError):
        c.check()
    assert torch.isfinite(got).all()


def test_refusals_of_the_c_abi():
    c = make(n_pages=4, page=16, kv=2, dim=64, rows=2, cols=2)
    s, off = dev([0]), dev([0, 1])
    x = torch.zeros((1, 2, 64), device="cuda")
    kv, p = c.kv, x.data_ptr()
    a = (s.data_ptr(), off.data_ptr())

    def with_(**kw):
        d = q.ovl_kv()
        for f, _ in q.ovl_kv._fields_:
            setattr(d, f, kw.get(f, getattr(kv, f)))
        return d

    for bad, st in ((dict(head_dim=96), q.OVL_E_SHAPE), (dict(page_tokens=24), q.OVL_E_SHAPE),
                    (dict(n_pages=0), q.OVL_E_SHAPE), (dict(n_layers=0), q.OVL_E_SHAPE),
                    (dict(n_kv_heads=0), q.OVL_E_SHAPE), (dict(max_seqs=0), q.OVL_E_SHAPE),
                    (dict(max_seqs=1 << 20), q.OVL_E_SHAPE), (dict(max_pages=1 << 30), q.OVL_E_SHAPE),
                    (dict(codes=0), q.OVL_E_ARG), (dict(scales=kv.scales + 8), q.OVL_E_SHAPE),
                    (dict(workspace=kv.workspace + 16), q.OVL_E_SHAPE), (dict(workspace_bytes=256), q.OVL_E_OOM)):
        assert q.ovl_kv_extend(with_(**bad), *a, 1) == st, bad
        assert q.ovl_last_error(None)
    ok = dict(layer=0, n=1, tokens=1, k=p, v=p, dt=q.OVL_F32, ks=128, vs=128)

    def append(**kw):
        d = {**ok, **kw}
        return q.ovl_kv_append(kv, d["layer"], *a, d["n"], d["tokens"], d["k"], d["v"], d["dt"], d["ks"], d["vs"])

    assert append(layer=1) == append(n=1025) == append(dt=3) == append(k=0) == q.OVL_E_ARG
    assert append(ks=64) == append(vs=130) == append(k=p + 4) == q.OVL_E_SHAPE
    assert append(n=0, k=0) == append(tokens=0, k=0) == q.OVL_OK
    ok2 = dict(layer=0, n=1, tokens=1, most=1, q=p, dt=q.OVL_F32, heads=2, qs=128, scale=1.0, out=p, os=128)

    def attend(**kw):
        d = {**ok2, **kw}
        return q.ovl_kv_attention(kv, d["layer"], *a, d["n"], d["tokens"], d["most"], d["q"], d["dt"], d["heads"],
                                  d["qs"], d["scale"], 0, 0, d["out"], d["os"])

    assert attend(layer=9) == attend(dt=0) == attend(scale=float("nan")) == attend(most=0) == q.OVL_E_ARG
    assert attend(q=0) == attend(out=0) == q.OVL_E_ARG
    assert attend(heads=3) == attend(heads=0) == attend(qs=100) == attend(out=p + 8) == attend(os=2) == q.OVL_E_SHAPE
    assert attend(n=0) == attend(tokens=0) == q.OVL_OK
    assert q.ovl_kv_read(kv, 0, *a, 1, 1, p, 0) == q.OVL_E_ARG
    assert q.ovl_kv_read(kv, 0, *a, 1, 1, p + 4, p) == q.OVL_E_SHAPE
    assert q.ovl_kv_fork(kv, a[0], 0, 0, 1) == q.OVL_E_ARG
    assert q.ovl_kv_compact(kv, a[0], a[0], 0, a[1], 1, 1) == q.OVL_E_ARG
    assert q.ovl_kv_release(kv, 0, 1) == q.OVL_E_ARG
    assert q.ovl_kv_release(kv, 0, 0) == q.OVL_OK
    assert q.ovl_kv_extend(None, *a, 1) == q.OVL_E_ARG
    c.check()


def test_refusals_of_the_torch_side():
    c = make(n_pages=4, page=16, kv=2, dim=64, rows=2, cols=2)
    s, off = dev([0]), dev([0, 1])
    x = torch.zeros((1, 2, 64), device="cuda")
    for bad in (x.half(), x[:, :1], x.cpu(), torch.zeros((1, 2, 128), device="cuda"),
                torch.zeros((1, 64, 2), device="cuda").transpose(1, 2)):
        with pytest.raises(ValueError):
            c.append(0, s, off, bad, x)
    with pytest.raises(ValueError):
        c.append(0, s.long(), off, x, x)
    with pytest.raises(ValueError):
        c.append(0, s, dev([0, 1, 2]), x, x)
    with pytest.raises(ValueError):
        c.attention(0, s, off, x, 1, out=x.bfloat16())
    with pytest.raises(q.OvlError):
        c.attention(0, s, off, torch.zeros((1, 3, 64), device="cuda"), 1)
    with pytest.raises(ValueError):
        KvCache(c.codes, c.scales[:, :, :1], c.table, c.length, c.refs)
    with pytest.raises(ValueError):
        KvCache(c.codes, c.scales, c.table.long(), c.length, c.refs)


def test_the_example_runs(capsys):
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decode_block.py")
    spec = importlib.util.spec_from_file_location("decode_block", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    m.main()
    said = capsys.readouterr().out
    assert "lengths: [307, 36, 305, 0]" in said and "after the release: 0" in said and "finite: True" in said

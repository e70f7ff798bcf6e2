"""A plain numpy statement of the 4-bit key/value cache, shared by its tests: the
block quantizer, where each code lies, attention in 64 bits, and the rows and
pages as lists.  It shares no code with the library."""
import numpy as np


def f16_of(x):
    return np.asarray(x, np.float32).astype(np.float16)


def quantize(x):
    """x float32 [..., D] -> codes uint8 [..., D], scales float16 [..., D / 32]."""
    b = np.asarray(x, np.float32).reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    b = np.where(np.isnan(b), np.float32(0), b)
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        d = f16_of(np.minimum(np.abs(b).max(-1) / np.float32(8), np.float32(65504)))
        t = b / d.astype(np.float32)[..., None]
        t = np.where(d.astype(np.float32)[..., None] > 0, t, np.float32(0))
        r = np.trunc(t + np.copysign(np.float32(0.5), t))
    code = (np.clip(r, -8, 7) + 8).astype(np.uint8)
    return code.reshape(x.shape), d


def values_of(codes, scales):
    return (codes.astype(np.float64) - 8) * np.repeat(scales.astype(np.float64), 32, axis=-1)


def key_address(slot, c, D):
    """(byte, low half?) of channel c of a token's key inside its unit."""
    block, word, at = c // 32, c % 32 // 8, c % 8
    return slot * (D // 2) + 4 * (word * (D // 32) + block) + at // 2, at % 2 == 0


def value_address(slot, c, D):
    unit, at = c % 8, c // 8
    return (slot // 8) * 4 * D + unit * (D // 2) + (slot % 8) * (D // 16) + at // 2, at % 2 == 0


def unpack(unit, page, D, which):
    """codes uint8 [page][D] of one unit's bytes."""
    out = np.empty((page, D), np.uint8)
    for slot in range(page):
        for c in range(D):
            byte, low = (key_address if which == 0 else value_address)(slot, c, D)
            out[slot, c] = unit[byte] & 15 if low else unit[byte] >> 4
    return out


def attention(q, k, v, positions, scale, window=0, sinks=0):
    """q [T][H][D], k and v [n][Hkv][D] (64-bit values), positions [T] -> (out [T][H][D], bound of its error per
    unit of relative error of the scores, largest |v| that the rows can weigh)."""
    T, H, D = q.shape
    n, hk = k.shape[0], k.shape[1]
    out, spread, top = np.zeros((T, H, D)), np.zeros((T, H, 1)), np.zeros((T, H, D))
    j, p = np.arange(n), np.asarray(positions)[:, None]
    seen = j <= p
    if window:
        seen &= (j > p - window) | (j < sinks)
    some = seen.any(1)
    if not some.any():
        return out, spread, top
    seen = seen[some]
    for h in range(H):
        kk, vv = k[:, h * hk // H], v[:, h * hk // H]
        s = np.where(seen, q[some, h] @ kk.T * scale, -np.inf)
        e = np.exp(s - s.max(1, keepdims=True))
        out[some, h] = (e / e.sum(1, keepdims=True)) @ vv
        spread[some, h, 0] = (np.where(seen, np.abs(q[some, h]) @ np.abs(kk).T, 0)).max(1) * abs(scale)
        top[some, h] = np.abs(vv[seen.any(0)]).max(0)
    return out, spread, top


def allowed(out, spread, top, bf16):
    """How far a result may be off.  A relative error e of every product of a score moves the score by at most
    e * spread, so each softmax weight by a factor 1 +- 2 e spread, and the output by 2 e spread top.
      float32: products good to 24 bits and 32-bit sums over at most 256 channels: e = 2^-20; exp, sums over the
               tokens and the division: 2^-19 top.
      bf16:    keys and queries rounded to 11 bits at most: e = 2^-11; the values' weights and the values rounded to
               11 bits each: 2^-10 top; the output to 8 bits: 2^-8 |out|."""
    if bf16:
        return (2 * 2.0 ** -11 * spread + 2.0 ** -10) * top + 2.0 ** -8 * np.abs(out) + 1e-30
    return (2 * 2.0 ** -20 * spread + 2.0 ** -19) * top + 1e-30


class Rows:
    """Rows, pages and reader counts as lists; a refused call raises and changes nothing."""

    def __init__(self, n_pages, page, max_seqs, max_pages):
        self.page, self.max_pages = page, max_pages
        self.refs = [0] * n_pages
        self.rows = [[] for _ in range(max_seqs)]
        self.length = [0] * max_seqs

    def _take(self, refs, count):
        free = [p for p, r in enumerate(refs) if r == 0][:count]
        if len(free) < count:
            raise MemoryError
        for p in free:
            refs[p] = 1
        return free

    def _distinct(self, dst, src=None):
        if len(set(dst)) != len(dst):
            raise KeyError
        if src is not None and any(s != d and s in set(dst) for s, d in zip(src, dst)):
            raise KeyError

    def extend(self, seqs, more):
        self._distinct(seqs)
        refs, new = list(self.refs), {}
        for s, m in zip(seqs, more):
            pages = -(-(self.length[s] + m) // self.page)
            if pages > self.max_pages:
                raise MemoryError
            new[s] = self.rows[s] + self._take(refs, pages - len(self.rows[s]))
        self.refs = refs
        for s, m in zip(seqs, more):
            self.rows[s] = new[s]
            self.length[s] += m

    def release(self, seqs):
        self._distinct(seqs)
        for s in seqs:
            for p in self.rows[s]:
                self.refs[p] -= 1
            self.rows[s], self.length[s] = [], 0

    def fork(self, src, dst, keep=None):
        self._distinct(dst, src)
        keep = [self.length[s] for s in src] if keep is None else keep
        refs, new = list(self.refs), []
        for s, d in zip(src, dst):
            if s != d:
                for p in self.rows[d]:
                    refs[p] -= 1
        for s, d, k in zip(src, dst, keep):
            if s != d:
                for p in self.rows[s][:k // self.page]:
                    refs[p] += 1
        late = []
        # in-place rows are judged before any page is handed out
        alone = [s == d and k % self.page and self.refs[self.rows[s][k // self.page]] == 1
                 for s, d, k in zip(src, dst, keep)]
        for s, d, k, mine in zip(src, dst, keep, alone):
            whole = k // self.page
            row = self.rows[s][:whole]
            if mine:
                row.append(self.rows[s][whole])
            elif k % self.page:
                row += self._take(refs, 1)
            if s == d:
                late += [p for p in self.rows[d] if p not in row]
            new.append(row)
        for p in late:
            refs[p] -= 1
        self.refs = refs
        for d, k, row in zip(dst, keep, new):
            self.rows[d], self.length[d] = row, k

    def compact(self, src, dst, counts):
        self._distinct(dst, src)
        refs, new = list(self.refs), []
        for s, d in zip(src, dst):
            if s != d:
                for p in self.rows[d]:
                    refs[p] -= 1
        for c in counts:
            new.append(self._take(refs, -(-c // self.page)))
        for s, d in zip(src, dst):
            if s == d:
                for p in self.rows[d]:
                    refs[p] -= 1
        self.refs = refs
        for d, c, row in zip(dst, counts, new):
            self.rows[d], self.length[d] = row, c

    def table(self):
        return np.array([r + [-1] * (self.max_pages - len(r)) for r in self.rows], np.int32)

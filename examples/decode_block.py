"""Attention of one decoder block over the 4-bit cache, next to the block's
quantized projections: a prompt, decode steps, two parallel samples, a rejected
draft taken back, and a context that is thinned out.

The block is the 8B shape (hidden 4096, 32 query heads and 8 kv heads of 128) with
seeded q8_0 projections; positions are rotated in torch.  Run from the repository's
root on the GPU, after the library is built:

    python examples/decode_block.py
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import numpy as np
import torch

import quantized_base_lora_gb300 as q
import synth as S
from quantized_base_lora_gb300.kvcache import KvCache
from quantized_base_lora_gb300.runtime import Runtime

HIDDEN, HEADS, KV, DIM = 4096, 32, 8, 128


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def rotate(x, pos):
    """Rotary positions: x [tokens][heads][DIM], pos [tokens]."""
    f = 10000.0 ** (-torch.arange(0, DIM, 2, device=x.device) / DIM)
    a = pos[:, None, None] * f
    u, v = x[..., 0::2], x[..., 1::2]
    return torch.stack((u * a.cos() - v * a.sin(), u * a.sin() + v * a.cos()), -1).flatten(-2)


class Block:
    def __init__(self, rows=4, pages=256):
        rng = np.random.default_rng(1)
        shapes = [(HEADS * DIM, HIDDEN), (KV * DIM, HIDDEN), (KV * DIM, HIDDEN), (HIDDEN, HEADS * DIM)]
        base = S.build_base(S.Q8_0, [(0, i, S.gaussian(rng, s, 0.02)) for i, s in enumerate(shapes)])
        self.rt = Runtime(arena_bytes=64 << 20)
        tensors = [(t.layer, t.proj, t.d_out, t.d_in, t.qs_off, t.d_off) for t in base.tensors]
        q.check(self.rt.load_base(base.quant, tensors, base.buf, S.content_digest(base.buf)), self.rt.ctx)
        self.cache = KvCache.allocate(n_pages=pages, page_tokens=64, n_layers=1, n_kv_heads=KV, head_dim=DIM,
                                      max_seqs=rows, max_pages=pages)
        self.length = [0] * rows                     # of each row, as the host knows it

    def step(self, seqs, counts, x):
        """The block's attention for counts[i] new tokens of row seqs[i]; x [tokens][HIDDEN], packed."""
        off = ints(np.concatenate([[0], np.cumsum(counts)]))
        rows = ints(seqs)
        pos = torch.cat([torch.arange(self.length[s], self.length[s] + n, device="cuda") for s, n in zip(seqs, counts)])
        parts = [self.rt.forward(i, x).unflatten(-1, (-1, DIM)) for i in range(3)]
        self.cache.extend(rows, off)
        self.cache.append(0, rows, off, rotate(parts[1], pos).bfloat16(), parts[2].bfloat16())
        o = self.cache.attention(0, rows, off, rotate(parts[0], pos).bfloat16(), max(counts))
        for s, n in zip(seqs, counts):
            self.length[s] += n
        return self.rt.forward(3, o.flatten(1))


def main():
    g = torch.Generator("cuda").manual_seed(0)
    b = Block()

    def tokens(n):
        return torch.randn((n, HIDDEN), generator=g, device="cuda").bfloat16()

    y = b.step([0, 1], [300, 77], tokens(377))                   # two prompts
    print("prompts:", tuple(y.shape))
    for _ in range(4):                                           # four decode steps of both
        y = b.step([0, 1], [1, 1], tokens(2))
    b.cache.fork(ints([0]), ints([2]))                           # a second sample of row 0 shares its full pages
    b.length[2] = b.length[0]
    y = b.step([0, 2], [1, 1], tokens(2))
    y = b.step([0], [5], tokens(5))                              # five drafted tokens, of which two are accepted
    b.length[0] -= 3
    b.cache.fork(ints([0]), ints([0]), ints([b.length[0]]))
    n = b.length[1]                                              # row 1 keeps its first 4 and its last 32 tokens
    keep = list(range(4)) + list(range(n - 32, n))
    b.cache.compact(ints([1]), ints([1]), ints(keep), ints([0, len(keep)]))
    print("lengths:", b.cache.length.tolist(), "pages in use:", int((b.cache.refs > 0).sum()))
    b.cache.release(ints([0, 1, 2]))
    b.cache.check()
    q.check(b.rt.check_device(), b.rt.ctx)
    print("pages in use after the release:", int((b.cache.refs > 0).sum()), "last output finite:",
          bool(torch.isfinite(y).all()))
    b.rt.close()


if __name__ == "__main__":
    main()

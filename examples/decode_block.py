"""One decoder block over the 4-bit cache, next to its quantized projections: a
prompt, decode steps, two parallel samples, a rejected draft taken back, and a
context that is thinned out.

The block's attention is the 8B shape (hidden 4096, 32 query heads and 8 kv heads of
128) with seeded q8_0 projections; behind it come a gated feed-forward part and a
mixture of experts, both small.  Norms, residuals, rotary positions, activations and
experts are the library's as well.  Run from the repository's root on the GPU, after
the library is built:

    python examples/decode_block.py
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import numpy as np
import torch

import quantized_base_lora_gb300 as q
import synth as S
from quantized_base_lora_gb300.block import BlockNorm, Moe, Norm, Rope, glu
from quantized_base_lora_gb300.kvcache import KvCache
from quantized_base_lora_gb300.runtime import Runtime

HIDDEN, HEADS, KV, DIM = 4096, 32, 8, 128
FFN, EXPERTS, TOP, EXPERT_FFN = 1024, 8, 2, 256


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Block:
    def __init__(self, rows=4, pages=256):
        rng = np.random.default_rng(1)
        shapes = [(HEADS * DIM, HIDDEN), (KV * DIM, HIDDEN), (KV * DIM, HIDDEN), (HIDDEN, HEADS * DIM),
                  (FFN, HIDDEN), (FFN, HIDDEN), (HIDDEN, FFN),
                  (EXPERTS * EXPERT_FFN, HIDDEN), (EXPERTS * EXPERT_FFN, HIDDEN), (EXPERTS * HIDDEN, EXPERT_FFN)]
        base = S.build_base(S.Q8_0, [(0, i, S.gaussian(rng, s, 0.02)) for i, s in enumerate(shapes)])
        self.rt = Runtime(arena_bytes=64 << 20)
        tensors = [(t.layer, t.proj, t.d_out, t.d_in, t.qs_off, t.d_off) for t in base.tensors]
        q.check(self.rt.load_base(base.quant, tensors, base.buf, S.content_digest(base.buf)), self.rt.ctx)
        self.cache = KvCache.allocate(n_pages=pages, page_tokens=64, n_layers=1, n_kv_heads=KV, head_dim=DIM,
                                      max_seqs=rows, max_pages=pages)
        self.rope = Rope(DIM, layout="pairs", base=500000.0, scaling="bands", factor=8.0, original=8192)
        w = [1 + 0.1 * torch.randn(HIDDEN, device="cuda") for _ in range(3)]
        self.norms = [BlockNorm(HIDDEN, Norm("rms", v)) for v in w] + [BlockNorm(HIDDEN, None)]
        self.moe = Moe.from_base(self.rt, 7, 8, 9, EXPERTS, TOP, max_tokens=128,
                                 router=torch.randn((EXPERTS, HIDDEN), device="cuda") * 0.02)

    def step(self, seqs, counts, x):
        """The block for counts[i] new tokens of row seqs[i]; x [tokens][HIDDEN], packed."""
        off = ints(np.concatenate([[0], np.cumsum(counts)]))
        rows, n = ints(seqs), sum(counts)
        self.cache.extend(rows, off)
        pos = self.cache.positions(rows, off, n)                     # once for all layers of a step
        x, h = self.norms[0](x)
        query, key, value = (self.rt.forward(i, h).unflatten(-1, (-1, DIM)) for i in range(3))
        query, key = self.rope(pos, query, key, dtype=torch.bfloat16)
        self.cache.append(0, rows, off, key, value.bfloat16())
        o = self.cache.attention(0, rows, off, query, max(counts))
        x, h = self.norms[1](x, self.rt.forward(3, o.flatten(1)))
        a = glu(self.rt.forward(4, h), self.rt.forward(5, h), dtype=torch.bfloat16)
        x, h = self.norms[2](x, self.rt.forward(6, a))
        y = torch.cat([self.moe(part) for part in h.split(self.moe.max_tokens)])
        return self.norms[3](x, y)[0]


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
    y = b.step([0, 2], [1, 1], tokens(2))
    y = b.step([0], [5], tokens(5))                              # five drafted tokens, of which two are accepted
    b.cache.fork(ints([0]), ints([0]), b.cache.length[:1] - 3)
    n = int(b.cache.length[1])                                   # row 1 keeps its first 4 and its last 32 tokens
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

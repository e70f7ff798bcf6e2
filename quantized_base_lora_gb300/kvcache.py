"""Torch-side convenience around the 4-bit key/value cache (ovl_kv_* in
include/ovl.h): holds the pools, the table and the workspace as torch tensors,
checks shapes and types, and passes addresses to the library.  PyTorch provides
device memory and streams only; all computation is libovl's.

    cache = KvCache.allocate(n_pages=4096, page_tokens=64, n_layers=32, n_kv_heads=8, head_dim=128,
                             max_seqs=64, max_pages=512)
    cache.extend(seqs, off)                        # once a step: pages for the new tokens
    for layer in range(32):
        cache.append(layer, seqs, off, k, v)       # k, v [tokens][kv heads][head_dim]
        o = cache.attention(layer, seqs, off, q, max_new)

Calls go to the current stream of the cache's device; calls on one cache must
be ordered by streams or events, since they share its workspace."""
from __future__ import annotations

import ctypes
import math

import torch

from . import (OVL_BF16, OVL_F32, OVL_OK, OvlError, lib, ovl_kv, ovl_kv_workspace_bytes, ovl_last_error)

_DTYPE = {torch.float32: OVL_F32, torch.bfloat16: OVL_BF16}


class KvCache:
    """codes uint8 [pages][layers][2][kv heads][page tokens * D / 2], scales float16 [pages][layers][2][kv heads]
    [page tokens][D / 32], table int32 [rows][columns], length int32 [rows], refs int32 [pages]: contiguous, on one
    CUDA device, kept by the cache and used as they are."""

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, table: torch.Tensor, length: torch.Tensor,
                 refs: torch.Tensor):
        if codes.dim() != 5 or scales.dim() != 6 or table.dim() != 2 or length.dim() != 1 or refs.dim() != 1:
            raise ValueError("codes [5 axes], scales [6], table [2], length [1] and refs [1] are wanted")
        pages, layers, two, heads, page, blocks = scales.shape
        dim = 32 * blocks
        if two != 2 or tuple(codes.shape) != (pages, layers, 2, heads, page * dim // 2):
            raise ValueError(f"codes {tuple(codes.shape)} and scales {tuple(scales.shape)} do not belong together")
        if refs.shape[0] != pages or length.shape[0] != table.shape[0]:
            raise ValueError("refs has one entry a page, length one a row of table")
        for name, t, dt in (("codes", codes, torch.uint8), ("scales", scales, torch.float16),
                            ("table", table, torch.int32), ("length", length, torch.int32),
                            ("refs", refs, torch.int32)):
            if t.dtype != dt or not t.is_contiguous() or t.device != codes.device or not t.is_cuda:
                raise ValueError(f"{name} must be a contiguous {dt} tensor on the cache's CUDA device")
        self.codes, self.scales, self.table, self.length, self.refs = codes, scales, table, length, refs
        self.device, self.n_kv_heads, self.head_dim, self.page_tokens = codes.device, heads, dim, page
        self.kv = ovl_kv(codes.data_ptr(), scales.data_ptr(), table.data_ptr(), length.data_ptr(), refs.data_ptr(),
                         None, 0, pages, page, layers, heads, dim, table.shape[0], table.shape[1])
        st, nbytes = ovl_kv_workspace_bytes(self.kv)
        self._check(st)
        self.workspace = torch.zeros(nbytes, dtype=torch.uint8, device=self.device)
        self.kv.workspace, self.kv.workspace_bytes = self.workspace.data_ptr(), nbytes
        self._at = ctypes.addressof(self.kv)

    @classmethod
    def allocate(cls, n_pages: int, page_tokens: int, n_layers: int, n_kv_heads: int, head_dim: int, max_seqs: int,
                 max_pages: int, device: int = 0) -> "KvCache":
        """An empty cache."""
        dev = torch.device("cuda", device)
        codes = torch.empty((n_pages, n_layers, 2, n_kv_heads, page_tokens * head_dim // 2), dtype=torch.uint8,
                            device=dev)
        scales = torch.empty((n_pages, n_layers, 2, n_kv_heads, page_tokens, head_dim // 32), dtype=torch.float16,
                             device=dev)
        self = cls(codes, scales, torch.empty((max_seqs, max_pages), dtype=torch.int32, device=dev),
                   torch.empty(max_seqs, dtype=torch.int32, device=dev),
                   torch.empty(n_pages, dtype=torch.int32, device=dev))
        with torch.cuda.device(dev):
            self._check(lib.ovl_kv_init(self._at, self._stream()))
        return self

    @staticmethod
    def _check(st: int):
        if st != OVL_OK:
            raise OvlError(st, ovl_last_error(None))

    def _stream(self) -> int:
        return torch.cuda.current_stream(self.device).cuda_stream

    def _ints(self, name: str, t: torch.Tensor, n: int | None = None) -> int:
        if t.dtype != torch.int32 or t.dim() != 1 or not t.is_contiguous() or t.device != self.device:
            raise ValueError(f"{name} must be a contiguous int32 vector on the cache's device")
        if n is not None and t.shape[0] != n:
            raise ValueError(f"{name} has {t.shape[0]} entries, {n} are wanted")
        return t.data_ptr()

    def _tokens(self, name: str, t: torch.Tensor, heads: int | None = None) -> int:
        """Address of packed tokens [tokens][heads][head_dim]; their stride is t.stride(0)."""
        if t.dim() != 3 or t.shape[2] != self.head_dim or (heads is not None and t.shape[1] != heads):
            raise ValueError(f"{name} {tuple(t.shape)} is not [tokens][{heads or 'heads'}][{self.head_dim}]")
        if t.dtype not in _DTYPE or t.device != self.device:
            raise ValueError(f"{name} must be float32 or bfloat16 on the cache's device")
        if t.stride(2) != 1 or (t.shape[1] > 1 and t.stride(1) != self.head_dim):
            raise ValueError(f"the heads and channels of {name} must be contiguous")
        return t.data_ptr()

    def _stride(self, t: torch.Tensor) -> int:
        return t.stride(0) if t.shape[0] > 1 else t.shape[1] * t.shape[2]

    def extend(self, seqs: torch.Tensor, tok_off: torch.Tensor):
        """Pages for tok_off[i+1] - tok_off[i] more tokens of row seqs[i]; length counts them."""
        n = seqs.shape[0]
        self._check(lib.ovl_kv_extend(self._at, self._ints("seqs", seqs), self._ints("tok_off", tok_off, n + 1), n,
                                      self._stream()))

    def append(self, layer: int, seqs: torch.Tensor, tok_off: torch.Tensor, k: torch.Tensor, v: torch.Tensor):
        """Write the last tokens of the rows: k, v [tokens][kv heads][head_dim] float32 or bfloat16."""
        n = seqs.shape[0]
        kp, vp = self._tokens("k", k, self.n_kv_heads), self._tokens("v", v, self.n_kv_heads)
        if k.dtype != v.dtype or k.shape[0] != v.shape[0]:
            raise ValueError("k and v must have one type and length")
        self._check(lib.ovl_kv_append(self._at, layer, self._ints("seqs", seqs), self._ints("tok_off", tok_off, n + 1),
                                      n, k.shape[0], kp, vp, _DTYPE[k.dtype], self._stride(k), self._stride(v),
                                      self._stream()))

    def read(self, layer: int, seqs: torch.Tensor, tok_off: torch.Tensor, n_tokens: int):
        """The values of the rows' last tokens: float32 (k, v), each [n_tokens][kv heads][head_dim]."""
        n = seqs.shape[0]
        out = torch.empty((2, n_tokens, self.n_kv_heads, self.head_dim), dtype=torch.float32, device=self.device)
        k, v = out[0], out[1]
        self._check(lib.ovl_kv_read(self._at, layer, self._ints("seqs", seqs), self._ints("tok_off", tok_off, n + 1),
                                    n, n_tokens, k.data_ptr(), v.data_ptr(), self._stream()))
        return k, v

    def attention(self, layer: int, seqs: torch.Tensor, tok_off: torch.Tensor, q: torch.Tensor, max_new: int,
                  scale: float | None = None, window: int = 0, sinks: int = 0,
                  out: torch.Tensor | None = None) -> torch.Tensor:
        """Attention of the rows' last tokens over the cache: q [tokens][heads][head_dim] -> the same shape and type.
        max_new: upper bound of the new tokens of one row; scale: 1 / sqrt(head_dim) unless given."""
        n = seqs.shape[0]
        qp = self._tokens("q", q)
        if out is None:
            out = torch.empty(q.shape, dtype=q.dtype, device=self.device)
        elif out.dtype != q.dtype or out.shape != q.shape:
            raise ValueError("out must have q's shape and type")
        if scale is None:
            scale = 1.0 / math.sqrt(self.head_dim)
        self._check(lib.ovl_kv_attention(self._at, layer, self._ints("seqs", seqs),
                                         self._ints("tok_off", tok_off, n + 1), n, q.shape[0], max_new, qp,
                                         _DTYPE[q.dtype], q.shape[1], self._stride(q), scale, window, sinks,
                                         self._tokens("out", out), self._stride(out), self._stream()))
        return out

    def fork(self, src: torch.Tensor, dst: torch.Tensor, keep: torch.Tensor | None = None):
        """Row dst[i] becomes the first keep[i] tokens of row src[i] (all without keep), sharing whole pages."""
        n = src.shape[0]
        self._check(lib.ovl_kv_fork(self._at, self._ints("src", src), self._ints("dst", dst, n),
                                    None if keep is None else self._ints("keep", keep, n), n, self._stream()))

    def compact(self, src: torch.Tensor, dst: torch.Tensor, keep: torch.Tensor, keep_off: torch.Tensor):
        """Row dst[i] becomes tokens keep[keep_off[i] .. keep_off[i+1] - 1] of row src[i], in fresh pages."""
        n = src.shape[0]
        self._check(lib.ovl_kv_compact(self._at, self._ints("src", src), self._ints("dst", dst, n),
                                       self._ints("keep", keep), self._ints("keep_off", keep_off, n + 1), n,
                                       keep.shape[0], self._stream()))

    def release(self, seqs: torch.Tensor):
        """The rows become free."""
        self._check(lib.ovl_kv_release(self._at, self._ints("seqs", seqs), seqs.shape[0], self._stream()))

    def check(self):
        """Wait for the current stream; raise what a call latched on the device since the last check."""
        self._check(lib.ovl_kv_check(self._at, self._stream()))

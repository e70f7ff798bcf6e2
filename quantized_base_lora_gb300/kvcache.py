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

Calls go to the current stream of the cache's device, whichever device is current;
calls on one cache must be ordered by streams or events, since they share its
workspace."""
from __future__ import annotations

import ctypes
import math

import torch

from . import (OVL_BF16, OVL_F32, OVL_OK, OvlError, lib, ovl_kv, ovl_kv_workspace_bytes, ovl_last_error)

_DTYPE = {torch.float32: OVL_F32, torch.bfloat16: OVL_BF16}


def _stream_of(index: int) -> int:
    return torch.cuda.current_stream(index).cuda_stream


# The current stream's handle without a Stream object around it (2 us a call less), where torch offers it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _stream_of)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


_U32 = 1 << 32      # numbers go to the library as 32 bits without a sign, where -1 would be the largest


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
        self._index, self._scale = codes.get_device(), 1.0 / math.sqrt(dim)
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
        self._call(lib.ovl_kv_init)
        return self

    @staticmethod
    def _check(st: int):
        if st != OVL_OK:
            raise OvlError(st, ovl_last_error(None))

    def _call(self, fn, *args):
        """fn(the cache, *args, stream) on the cache's device (the library launches on the current one)."""
        if _current_device() == self._index:
            st = fn(self._at, *args, _raw_stream(self._index))
        else:
            with torch.cuda.device(self._index):
                st = fn(self._at, *args, _raw_stream(self._index))
        if st:
            self._check(st)

    # The checks below run at every call, for every tensor: they read each property once.

    def _ints(self, name: str, t: torch.Tensor, n: int) -> int:
        """Address of an int32 vector of n entries."""
        if t.dtype is not torch.int32 or t.shape != (n,) or not t.is_contiguous() or t.get_device() != self._index:
            raise ValueError(f"{name} must be a contiguous int32 vector of {n} entries on the cache's device, not "
                             f"{t.dtype} {tuple(t.shape)} on {t.device}")
        return t.data_ptr()

    def _tokens(self, name: str, t: torch.Tensor, heads: int | None = None):
        """(address, tokens, heads, dtype code, stride) of packed tokens [tokens][heads][head_dim]."""
        if t.dim() != 3:
            raise ValueError(f"{name} {tuple(t.shape)} is not [tokens][heads][{self.head_dim}]")
        n, h, d = t.shape
        step, by_head, by_channel = t.stride()
        code = _DTYPE.get(t.dtype)
        if d != self.head_dim or (heads is not None and h != heads):
            raise ValueError(f"{name} {tuple(t.shape)} is not [tokens][{heads or 'heads'}][{self.head_dim}]")
        if code is None or t.get_device() != self._index:
            raise ValueError(f"{name} must be float32 or bfloat16 on the cache's device")
        if by_channel != 1 or (h > 1 and by_head != d):
            raise ValueError(f"the heads and channels of {name} must be contiguous")
        return t.data_ptr(), n, h, code, (step if n > 1 else h * d)

    def extend(self, seqs: torch.Tensor, tok_off: torch.Tensor):
        """Pages for tok_off[i+1] - tok_off[i] more tokens of row seqs[i]; length counts them."""
        n = seqs.shape[0]
        self._call(lib.ovl_kv_extend, self._ints("seqs", seqs, n), self._ints("tok_off", tok_off, n + 1), n)

    def append(self, layer: int, seqs: torch.Tensor, tok_off: torch.Tensor, k: torch.Tensor, v: torch.Tensor):
        """Write the last tokens of the rows: k, v [tokens][kv heads][head_dim] float32 or bfloat16."""
        if not 0 <= layer < _U32:
            raise ValueError(f"layer {layer} is out of range")
        n = seqs.shape[0]
        kp, tokens, _, code, ks = self._tokens("k", k, self.n_kv_heads)
        vp, v_tokens, _, v_code, vs = self._tokens("v", v, self.n_kv_heads)
        if code != v_code or tokens != v_tokens:
            raise ValueError("k and v must have one type and length")
        self._call(lib.ovl_kv_append, layer, self._ints("seqs", seqs, n), self._ints("tok_off", tok_off, n + 1), n,
                   tokens, kp, vp, code, ks, vs)

    def read(self, layer: int, seqs: torch.Tensor, tok_off: torch.Tensor, n_tokens: int):
        """The values of the rows' last tokens: float32 (k, v), each [n_tokens][kv heads][head_dim]."""
        if not (0 <= layer < _U32 and 0 <= n_tokens < _U32):
            raise ValueError(f"layer {layer} or n_tokens {n_tokens} is out of range")
        n = seqs.shape[0]
        k = torch.empty((n_tokens, self.n_kv_heads, self.head_dim), dtype=torch.float32, device=self.device)
        v = torch.empty_like(k)
        if n == 0:                                   # no sequence, so no call: tokens that no one owns are zeros
            return k.zero_(), v.zero_()
        self._call(lib.ovl_kv_read, layer, self._ints("seqs", seqs, n), self._ints("tok_off", tok_off, n + 1), n,
                   n_tokens, k.data_ptr(), v.data_ptr())
        return k, v

    def attention(self, layer: int, seqs: torch.Tensor, tok_off: torch.Tensor, q: torch.Tensor, max_new: int,
                  scale: float | None = None, window: int = 0, sinks: int = 0,
                  out: torch.Tensor | None = None) -> torch.Tensor:
        """Attention of the rows' last tokens over the cache: q [tokens][heads][head_dim] -> the same shape and type.
        max_new: upper bound of the new tokens of one row; scale: 1 / sqrt(head_dim) unless given."""
        if not (0 <= layer < _U32 and 0 <= max_new < _U32 and 0 <= window < _U32 and 0 <= sinks < _U32):
            raise ValueError(f"layer {layer}, max_new {max_new}, window {window} or sinks {sinks} is out of range")
        n = seqs.shape[0]
        qp, tokens, heads, code, qs = self._tokens("q", q)
        if out is None:
            out = torch.empty_like(q, memory_format=torch.contiguous_format)
            op, os_ = out.data_ptr(), heads * self.head_dim
        else:
            op, o_tokens, o_heads, o_code, os_ = self._tokens("out", out)
            if (o_tokens, o_heads, o_code) != (tokens, heads, code):
                raise ValueError("out must have q's shape and type")
        if n == 0:
            return out.zero_()
        self._call(lib.ovl_kv_attention, layer, self._ints("seqs", seqs, n), self._ints("tok_off", tok_off, n + 1), n,
                   tokens, max_new, qp, code, heads, qs, self._scale if scale is None else scale, window, sinks, op, os_)
        return out

    def fork(self, src: torch.Tensor, dst: torch.Tensor, keep: torch.Tensor | None = None):
        """Row dst[i] becomes the first keep[i] tokens of row src[i] (all without keep), sharing whole pages."""
        n = src.shape[0]
        self._call(lib.ovl_kv_fork, self._ints("src", src, n), self._ints("dst", dst, n),
                   None if keep is None else self._ints("keep", keep, n), n)

    def compact(self, src: torch.Tensor, dst: torch.Tensor, keep: torch.Tensor, keep_off: torch.Tensor):
        """Row dst[i] becomes tokens keep[keep_off[i] .. keep_off[i+1] - 1] of row src[i], in fresh pages."""
        n = src.shape[0]
        m = keep.shape[0]
        self._call(lib.ovl_kv_compact, self._ints("src", src, n), self._ints("dst", dst, n), self._ints("keep", keep, m),
                   self._ints("keep_off", keep_off, n + 1), n, m)

    def release(self, seqs: torch.Tensor):
        """The rows become free."""
        n = seqs.shape[0]
        self._call(lib.ovl_kv_release, self._ints("seqs", seqs, n), n)

    def check(self):
        """Wait for the current stream; raise what a call latched on the device since the last check."""
        self._call(lib.ovl_kv_check)

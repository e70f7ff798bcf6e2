"""Torch-side convenience around what a decoder block computes between its projections
(ovl_rope_apply, ovl_block_norm_apply, ovl_glu and ovl_moe_forward in include/ovl.h).
PyTorch provides device memory and streams only; all computation is libovl's.

    rope = Rope(128, base=500000.0, scaling="bands", factor=8.0, original=8192)
    norm = BlockNorm(4096, Norm("rms", w))
    x, h = norm(x, y)                                  # x + y, and its norm for the next block
    q, k = rope(pos, q, k, dtype=torch.bfloat16)       # pos: cache.positions(seqs, off, tokens)
    a = glu(gate, up, dtype=torch.bfloat16)
    y = moe(h)                                         # Moe(...): router, chosen experts, weighted sum

Calls go to the current stream of the tensors' device, whichever device is current; those of one Moe must be
ordered by streams or events, since they share its workspace.  Tensors are float32 or
bfloat16 with contiguous channels; tokens may have any stride that is not below their width (an expanded row is
refused).  Nothing is differentiated."""
from __future__ import annotations

import ctypes
import struct
from typing import NamedTuple

import torch

from . import (OVL_ACT_GELU, OVL_ACT_GELU_TANH, OVL_ACT_RELU, OVL_ACT_SILU, OVL_E_STATE, OVL_F32, OVL_MOE_SIGMOID,
               OVL_MOE_SOFTMAX, OVL_NORM_LAYER, OVL_NORM_NONE, OVL_NORM_RMS, OVL_OK, OVL_PACKED_BLOCK_NORM, OVL_PACKED_GLU,
               OVL_PACKED_MOE, OVL_PACKED_ROPE, OVL_Q8_0, OVL_ROPE_BANDS, OVL_ROPE_BASE, OVL_ROPE_HALF,
               OVL_ROPE_LINEAR, OVL_ROPE_PAIRS, OVL_ROPE_PLAIN, OVL_ROPE_RAMP, OvlError, check, lib,
               ovl_block_norm, ovl_count_overlays, ovl_last_error, ovl_moe, ovl_moe_workspace_bytes, ovl_norm, ovl_rope)
from .kvcache import _DTYPE, _current_device, _raw_stream

_LAYOUT = {"half": OVL_ROPE_HALF, "pairs": OVL_ROPE_PAIRS}
_SCALING = {None: OVL_ROPE_PLAIN, "none": OVL_ROPE_PLAIN, "linear": OVL_ROPE_LINEAR, "base": OVL_ROPE_BASE,
            "bands": OVL_ROPE_BANDS, "ramp": OVL_ROPE_RAMP}
_TURNS = {"bands": (1.0, 4.0), "ramp": (1.0, 32.0)}      # low and high, unless given
_NORM = {None: OVL_NORM_NONE, "rms": OVL_NORM_RMS, "layer": OVL_NORM_LAYER}
_ACT = {"silu": OVL_ACT_SILU, "gelu": OVL_ACT_GELU, "gelu_tanh": OVL_ACT_GELU_TANH, "relu": OVL_ACT_RELU}
_SCORE = {"softmax": OVL_MOE_SOFTMAX, "sigmoid": OVL_MOE_SIGMOID}
_MOST = (1 << 31) - 1
_packed = lib.ovl_packed
_address = ctypes.addressof
_FLAT = torch.contiguous_format


def _check(st: int):
    if st != OVL_OK:
        raise OvlError(st, ovl_last_error(None))


# The library's calls take their arguments as one string of 64-bit words: ctypes converts
# each argument of a call by itself, 1.9 us for a norm's instead of 0.5.
_words11, _words15, _words18 = (struct.Struct(f"={n}Q").pack for n in (11, 15, 18))


def _call(index: int, which: int, words: bytes):
    """The packed call on device `index`, on its current stream (the library launches on the current device)."""
    if _current_device() == index:
        st = _packed(which, words, len(words) >> 3, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            st = _packed(which, words, len(words) >> 3, _raw_stream(index))
    if st:
        _check(st)


def _named(table: dict, name: str, value):
    code = table.get(value)
    if code is None:
        raise ValueError(f"{name} must be one of {[k for k in table if k is not None]}, not {value!r}")
    return code


# The checks below run at every call, for every tensor: they read each property once.

def _rows(name: str, t: torch.Tensor, width: int, index: int):
    """(address, tokens, dtype code, stride) of [tokens][width]."""
    shape = t.shape
    if len(shape) != 2 or shape[1] != width:
        raise ValueError(f"{name} {tuple(shape)} is not [tokens][{width}]")
    step, by_channel = t.stride()
    code = _DTYPE.get(t.dtype)
    if code is None or t.get_device() != index:
        raise ValueError(f"{name} must be float32 or bfloat16 on cuda:{index}, not {t.dtype} on {t.device}")
    if by_channel != 1 and width > 1:
        raise ValueError(f"the channels of {name} must be contiguous")
    n = shape[0]
    return t.data_ptr(), n, code, (step if n > 1 else width)


def _out(name: str, t: torch.Tensor, n: int, width: int, code: int, index: int):
    """(address, stride) of an output tensor that the caller gave."""
    p, m, c, s = _rows(name, t, width, index)
    if m != n or c != code:
        raise ValueError(f"{name} {tuple(t.shape)} of {t.dtype} is not the output's shape and type")
    return p, s


def _index_of(name: str, t: torch.Tensor) -> int:
    index = t.get_device()
    if index < 0:
        raise ValueError(f"{name} must be on a CUDA device, not {t.device}")
    return index


def _ints(name: str, t: torch.Tensor, shape: tuple, index: int) -> int:
    if t.dtype is not torch.int32 or t.shape != shape or not t.is_contiguous() or t.get_device() != index:
        raise ValueError(f"{name} must be contiguous int32 {shape} on cuda:{index}, not {t.dtype} {tuple(t.shape)} on "
                         f"{t.device}")
    return t.data_ptr()


class Rope:
    """Rotary positions of the first rot_dim channels of heads of head_dim; see ovl_rope_plan for the scalings.
    layout "half": channel i turns with i + rot_dim / 2; "pairs": 2 i with 2 i + 1."""

    def __init__(self, head_dim: int, rot_dim: int | None = None, layout: str = "half", base: float = 10000.0,
                 scaling: str | None = None, factor: float = 1.0, original: int = 0, low: float | None = None,
                 high: float | None = None, magnitude: float | None = None):
        rot_dim = head_dim if rot_dim is None else rot_dim
        if not (0 <= head_dim <= _MOST and 0 <= rot_dim <= _MOST and 0 <= original <= _MOST):
            raise ValueError("head_dim, rot_dim or original is out of range")
        kind = _named(_SCALING, "scaling", scaling)
        turns = _TURNS.get(scaling, (1.0, 2.0))
        self.head_dim, self.plan = head_dim, ovl_rope()
        _check(lib.ovl_rope_plan(head_dim, rot_dim, _named(_LAYOUT, "layout", layout), base, kind, factor, original,
                                 turns[0] if low is None else low, turns[1] if high is None else high,
                                 0.0 if magnitude is None else magnitude, ctypes.byref(self.plan)))

    def _heads(self, name: str, t: torch.Tensor, index: int):
        """(address, tokens, heads, dtype code, stride) of [tokens][heads][head_dim]."""
        shape, d = t.shape, self.head_dim
        if len(shape) != 3 or shape[2] != d:
            raise ValueError(f"{name} {tuple(shape)} is not [tokens][heads][{d}]")
        n, h, _ = shape
        step, by_head, by_channel = t.stride()
        code = _DTYPE.get(t.dtype)
        if code is None or t.get_device() != index:
            raise ValueError(f"{name} must be float32 or bfloat16 on cuda:{index}, not {t.dtype} on {t.device}")
        if by_channel != 1 or (h > 1 and by_head != d):
            raise ValueError(f"the heads and channels of {name} must be contiguous")
        return t.data_ptr(), n, h, code, (step if n > 1 else h * d)

    def __call__(self, pos: torch.Tensor, q: torch.Tensor, k: torch.Tensor | None = None,
                 dtype: torch.dtype | None = None, q_out: torch.Tensor | None = None,
                 k_out: torch.Tensor | None = None):
        """q, and k where given, turned to pos (int32 [tokens]): [tokens][heads][head_dim] in dtype (q's unless given).
        q_out and k_out may be q and k themselves.  Returns q', or (q', k')."""
        index = _index_of("q", q)
        qp, n, qh, code, qs = self._heads("q", q, index)
        dtype = q.dtype if dtype is None else dtype
        out_code = _DTYPE.get(dtype)
        if out_code is None:
            raise ValueError(f"dtype must be float32 or bfloat16, not {dtype}")
        if q_out is None:
            q_out = torch.empty_like(q, dtype=dtype, memory_format=_FLAT)
            qop, qos = q_out.data_ptr(), qh * self.head_dim
        else:
            qop, m, h, c, qos = self._heads("q_out", q_out, index)
            if (m, h, c) != (n, qh, out_code):
                raise ValueError("q_out must have q's shape and the output's type")
        kp = kh = ks = kop = kos = 0
        if k is not None:
            kp, m, kh, c, ks = self._heads("k", k, index)
            if m != n or c != code:
                raise ValueError("q and k must have one type and length")
            if k_out is None:
                k_out = torch.empty_like(k, dtype=dtype, memory_format=_FLAT)
                kop, kos = k_out.data_ptr(), kh * self.head_dim
            else:
                kop, m, h, c, kos = self._heads("k_out", k_out, index)
                if (m, h, c) != (n, kh, out_code):
                    raise ValueError("k_out must have k's shape and the output's type")
        elif k_out is not None:
            raise ValueError("k_out without k")
        if n > _MOST:
            raise ValueError("too many tokens")
        # the plan's address is taken here: a copy of this object has a plan of its own
        _call(index, OVL_PACKED_ROPE, _words15(_address(self.plan), n, _ints("pos", pos, (n,), index), qp, qh, qs, kp, kh,
                                               ks, code, qop, qos, kop, kos, out_code))
        return q_out if k is None else (q_out, k_out)


class Norm(NamedTuple):
    """One norm: kind "rms" or "layer", weight and bias [hidden] or None; offset is added to the weight."""
    kind: str
    weight: torch.Tensor | None = None
    bias: torch.Tensor | None = None
    eps: float = 1e-6
    offset: float = 0.0


class BlockNorm:
    """x' = alpha x + beta gate * post(y), h = pre(x'): the end of one block and the beginning of the next.  Weights and
    biases are used where they lie at construction: writes into them count, another storage (`w.data = ...`, as
    Module.to sets it) does not."""

    def __init__(self, hidden: int, pre: Norm | None, post: Norm | None = None, alpha: float = 1.0, beta: float = 1.0):
        if not 0 <= hidden <= _MOST:
            raise ValueError(f"hidden {hidden} is out of range")
        self.hidden, self.pre, self.post, self._index, self._held = hidden, pre, post, None, []
        self.plan = ovl_block_norm(hidden, alpha, beta, self._norm("post", post), self._norm("pre", pre))
        self._at = ctypes.addressof(self.plan)

    def _norm(self, name: str, n: Norm | None) -> ovl_norm:
        if n is None:
            return ovl_norm(OVL_NORM_NONE, OVL_F32, None, None, 0.0, 0.0)
        at, code = [], OVL_F32
        for what, t in (("weight", n.weight), ("bias", n.bias)):
            if t is None:
                at.append(None)
                continue
            index = _index_of(f"{name}.{what}", t)
            if self._index is not None and index != self._index:
                raise ValueError("weights and biases must be on one device")
            self._index = index
            if t.shape != (self.hidden,) or not t.is_contiguous() or t.dtype not in _DTYPE:
                raise ValueError(f"{name}.{what} must be contiguous float32 or bfloat16 [{self.hidden}]")
            code = _DTYPE[t.dtype]
            at.append(t.data_ptr())
            self._held.append(t.detach())                # the storage, whatever becomes of the tensor's
        if n.weight is not None and n.bias is not None and n.weight.dtype != n.bias.dtype:
            raise ValueError(f"weight and bias of {name} must have one type")
        return ovl_norm(_named(_NORM, "kind", n.kind), code, at[0], at[1], n.eps, n.offset)

    def __call__(self, x: torch.Tensor, y: torch.Tensor | None = None, gate: torch.Tensor | None = None,
                 gate_row: torch.Tensor | None = None, dtype: torch.dtype | None = None,
                 x_out: torch.Tensor | None = None, h_out: torch.Tensor | None = None):
        """x, y [tokens][hidden] -> (x' in x's type, h in dtype, x's unless given; None without a pre norm).
        gate: [hidden], [rows][hidden] with gate_row int32 [tokens], or [tokens][hidden].  x_out may be x."""
        index = _index_of("x", x)
        if self._index is not None and index != self._index:
            raise ValueError(f"x is on cuda:{index}, the norms' weights on cuda:{self._index}")
        hidden = self.hidden
        xp, n, x_code, xs = _rows("x", x, hidden, index)
        yp = ys = 0
        y_code = OVL_F32
        if y is not None:
            yp, m, y_code, ys = _rows("y", y, hidden, index)
            if m != n:
                raise ValueError("x and y must have one length")
        gp = gs = rows = rp = 0
        g_code = OVL_F32
        if gate is not None:
            if y is None:
                raise ValueError("gate without y")
            gp, rows, g_code, gs = _rows("gate", gate.unsqueeze(0) if gate.dim() == 1 else gate, hidden, index)
            if gate_row is not None:
                rp = _ints("gate_row", gate_row, (n,), index)
            elif rows not in (1, n):
                raise ValueError("without gate_row there is one gate, or one for each token")
            if rows == 0:
                raise ValueError("gate has no rows")
        elif gate_row is not None:
            raise ValueError("gate_row without gate")
        if x_out is None:
            x_out = torch.empty_like(x, memory_format=_FLAT)
            xop, xos = x_out.data_ptr(), hidden
        else:
            xop, xos = _out("x_out", x_out, n, hidden, x_code, index)
        dtype = x.dtype if dtype is None else dtype
        h_code = _DTYPE.get(dtype)
        if h_code is None:
            raise ValueError(f"dtype must be float32 or bfloat16, not {dtype}")
        hp = hs = 0
        if self.pre is None:
            if h_out is not None:
                raise ValueError("h_out without a pre norm")
        elif h_out is None:
            h_out = torch.empty_like(x, dtype=dtype, memory_format=_FLAT)
            hp, hs = h_out.data_ptr(), hidden
        else:
            hp, hs = _out("h_out", h_out, n, hidden, h_code, index)
        if n == 0:
            return x_out, h_out
        if n > _MOST or rows > _MOST:
            raise ValueError("too many tokens or gates")
        _call(index, OVL_PACKED_BLOCK_NORM, _words18(self._at, n, xp, x_code, xs, yp, y_code, ys, gp, g_code, gs, rp,
                                                     rows, xop, xos, hp, h_code, hs))
        return x_out, h_out


def glu(gate: torch.Tensor, up: torch.Tensor, act: str = "silu", dtype: torch.dtype | None = None,
        out: torch.Tensor | None = None) -> torch.Tensor:
    """act(gate) * up: [tokens][width] in dtype (gate's unless given).  out may be gate or up."""
    index = _index_of("gate", gate)
    width = gate.shape[-1]
    gp, n, code, gs = _rows("gate", gate, width, index)
    up_, m, c, us = _rows("up", up, width, index)
    if m != n or c != code:
        raise ValueError("gate and up must have one type and shape")
    dtype = gate.dtype if dtype is None else dtype
    out_code = _DTYPE.get(dtype)
    if out_code is None:
        raise ValueError(f"dtype must be float32 or bfloat16, not {dtype}")
    if out is None:
        out = torch.empty_like(gate, dtype=dtype, memory_format=_FLAT)
        op, os_ = out.data_ptr(), width
    else:
        op, os_ = _out("out", out, n, width, out_code, index)
    if n > _MOST or width > _MOST:
        raise ValueError("too many tokens or channels")
    _call(index, OVL_PACKED_GLU, _words11(_named(_ACT, "act", act), n, width, gp, gs, up_, us, code, op, os_, out_code))
    return out


def _refuse_overlays(runtime, tensors):
    if runtime.ctx:                                      # closed: no composition, and the base's planes are kept
        st, n = ovl_count_overlays(runtime.ctx, tensors)
        check(st, runtime.ctx)
        if n:
            raise OvlError(OVL_E_STATE, f"the active composition overlays an expert tensor (of {tensors}), and overlays "
                                        "are not applied to experts")


class Moe:
    """A mixture-of-experts layer over quantized experts, for up to max_tokens (at most 128) tokens a call.

    gate, up: (qs, d) of [n_experts * ffn] rows of hidden weights, down: of [n_experts * hidden] rows of ffn weights, in
    the base's layout of `quant`: qs int8 or uint8 and d float16 (q4_K: uint8) tensors, contiguous, of any shape with
    the right number of bytes.  They must not be written while calls that read them are in flight.  router
    [n_experts][hidden], bias float32 [n_experts]; without a router every call brings its choice.  All are used where
    they lie at construction, as BlockNorm's weights are.

    Calls on one layer must be ordered by streams or events, replays of graphs that hold them included, since they
    share its workspace; layers of their own may run beside one another."""

    def __init__(self, quant: int, n_experts: int, hidden: int, ffn: int, gate, up, down, top_k: int,
                 router: torch.Tensor | None = None, bias: torch.Tensor | None = None, score: str = "softmax",
                 renormalize: bool = True, scale: float = 1.0, act: str = "silu", max_tokens: int = 64):
        for name, v in (("quant", quant), ("n_experts", n_experts), ("hidden", hidden), ("ffn", ffn), ("top_k", top_k),
                        ("max_tokens", max_tokens)):
            if not 0 <= v <= _MOST:
                raise ValueError(f"{name} {v} is out of range")
        self.moe = ovl_moe(quant, n_experts, top_k, hidden, ffn, _named(_ACT, "act", act),
                           _named(_SCORE, "score", score), bool(renormalize), scale, OVL_F32, max_tokens)
        st, nbytes = ovl_moe_workspace_bytes(self.moe)
        _check(st)
        self._index = _index_of("gate", gate[0])
        self.device, self.hidden, self.top_k, self.max_tokens = gate[0].device, hidden, top_k, max_tokens
        weights = n_experts * hidden * ffn
        for name, planes in (("gate", gate), ("up", up), ("down", down)):
            for part, t, need in (("qs", planes[0], weights if quant == OVL_Q8_0 else weights // 2),
                                  ("d", planes[1], weights // 16)):
                if t.get_device() != self._index or not t.is_contiguous() or t.numel() * t.element_size() != need:
                    raise ValueError(f"{name}'s {part} plane must be contiguous, {need} bytes, on one CUDA device")
                setattr(self.moe, f"{name}_{part}", t.data_ptr())
        if router is not None:
            if router.shape != (n_experts, hidden) or not router.is_contiguous() or router.get_device() != self._index \
                    or router.dtype not in _DTYPE:
                raise ValueError(f"router must be contiguous float32 or bfloat16 [{n_experts}][{hidden}]")
            self.moe.router, self.moe.router_dtype = router.data_ptr(), _DTYPE[router.dtype]
        if bias is not None:
            if bias.shape != (n_experts,) or not bias.is_contiguous() or bias.get_device() != self._index \
                    or bias.dtype != torch.float32:
                raise ValueError(f"bias must be contiguous float32 [{n_experts}]")
            self.moe.bias = bias.data_ptr()
        # the storages, whatever becomes of the tensors'
        self._held = (*((p[0].detach(), p[1].detach()) for p in (gate, up, down)),
                      *(None if t is None else t.detach() for t in (router, bias)))
        self.workspace = torch.zeros(nbytes, dtype=torch.uint8, device=self.device)
        self.moe.workspace, self.moe.workspace_bytes = self.workspace.data_ptr(), nbytes
        self._at = ctypes.addressof(self.moe)
        self._runtime = self._tensors = None

    @classmethod
    def from_base(cls, runtime, gate: int, up: int, down: int, n_experts: int, top_k: int, **more) -> "Moe":
        """Experts that are tensors of a loaded base: gate and up have n_experts * ffn rows of hidden weights, down
        n_experts * hidden rows of ffn weights.  Overlays are not applied to experts: a call raises (OVL_E_STATE) while the
        runtime's active composition has one on any of the three.  (Replays of a captured call are not asked.)"""
        quant = runtime.quant
        planes = []
        for i in (gate, up, down):
            _, _, rows, columns, qs, d = runtime.tensors[i]
            n = rows * columns
            planes.append((runtime.base[qs:qs + (n if quant == OVL_Q8_0 else n // 2)], runtime.base[d:d + n // 16]))
        hidden = runtime.tensors[gate][3]
        ffn = runtime.tensors[down][3]
        for i, want in ((gate, (n_experts * ffn, hidden)), (up, (n_experts * ffn, hidden)),
                        (down, (n_experts * hidden, ffn))):
            if tuple(runtime.tensors[i][2:4]) != want:
                raise ValueError(f"tensor {i} is {tuple(runtime.tensors[i][2:4])}, not {want}")
        tensors = tuple(range(len(runtime.tensors))[i] for i in (gate, up, down))
        _refuse_overlays(runtime, tensors)
        layer = cls(quant, n_experts, hidden, ffn, *planes, top_k, **more)
        layer._runtime, layer._tensors = runtime, tensors
        return layer

    def __call__(self, x: torch.Tensor, choice: torch.Tensor | None = None, weight: torch.Tensor | None = None,
                 out: torch.Tensor | None = None, routing: bool = False):
        """x [tokens][hidden] -> y of the same shape and type; with routing (y, choice int32, weight float32).
        choice int32 and weight float32 [tokens][top_k] take the router's place; a negative choice is none."""
        if self._runtime is not None:
            _refuse_overlays(self._runtime, self._tensors)
        index = self._index
        xp, n, code, xs = _rows("x", x, self.hidden, index)
        if n > self.max_tokens:
            raise ValueError(f"{n} tokens, max_tokens is {self.max_tokens}")
        if out is None:
            out = torch.empty_like(x, memory_format=_FLAT)
            op, os_ = out.data_ptr(), self.hidden
        else:
            op, os_ = _out("out", out, n, self.hidden, code, index)
        shape = (n, self.top_k)
        cp = wp = cop = wop = 0
        if (choice is None) != (weight is None):
            raise ValueError("choice and weight come together")
        if choice is not None:
            cp = _ints("choice", choice, shape, index)
            if weight.dtype is not torch.float32 or weight.shape != shape or not weight.is_contiguous() \
                    or weight.get_device() != index:
                raise ValueError(f"weight must be contiguous float32 {shape} on cuda:{index}")
            wp = weight.data_ptr()
            if routing:
                raise ValueError("routing returns the router's choice, and the choice is given")
        if routing:
            choice_out = torch.empty(shape, dtype=torch.int32, device=x.device)
            weight_out = torch.empty(shape, dtype=torch.float32, device=x.device)
            cop, wop = choice_out.data_ptr(), weight_out.data_ptr()
        if n:
            _call(index, OVL_PACKED_MOE, _words11(self._at, xp, code, n, xs, cp, wp, cop, wop, op, os_))
        return (out, choice_out, weight_out) if routing else out

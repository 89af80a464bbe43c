"""Linear attention with a decay for each head (include/moe_block.h) over torch
tensors: the layers of a hybrid decoder that keep a state instead of a cache.

`LinearAttention` holds one layer's states, [n_slots][Hv][Dk][Dv] fp32, and
forwards calls to libmoe_gb300.so. A program empties a slot with
`states.state[slot] = 0` and forks one with `states.state[dst] = states.state[src]`.

    o = states.step(q, k, v, g, slots=slots)                        # a token per slot
    o = states.chunk(q, k, v, g, slots=slots, row_start=row_start)  # prompts
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib
from ._lib import MOE_KV_BF16, MOE_KV_F16, moe_kv_rows, moe_linear_args, moe_linear_desc
from .block import _new, _on

_DTYPES = {torch.bfloat16: MOE_KV_BF16, torch.float16: MOE_KV_F16}
_I32, _F32 = torch.int32, torch.float32


class LinearAttention:
    """State of one layer: Hk heads of queries and keys of Dk values, shared in groups by
    Hv heads of values of Dv; q, k, v and o in `dtype`. A call works on the current
    stream, or on `stream` (a torch stream or a handle), whose the results are then;
    ordering it with other streams, and keeping the arguments alive until it has run,
    is the caller's. Calls on the same slots must be ordered; others need not be."""

    def __init__(self, n_slots, Hk, Hv, Dk, Dv, dtype=torch.bfloat16, device="cuda"):
        self._setup(torch.zeros(n_slots, Hv, Dk, Dv, dtype=_F32, device=device), Hk, dtype)

    @classmethod
    def over(cls, state, Hk, dtype=torch.bfloat16):
        """Over the caller's states (used in place)."""
        self = cls.__new__(cls)
        self._setup(state, Hk, dtype)
        return self

    def _setup(self, state, Hk, dtype):
        if state.dim() != 4 or state.dtype != _F32 or not state.is_contiguous():
            raise ValueError("state must be a contiguous fp32 [n_slots][Hv][Dk][Dv]")
        if dtype not in _DTYPES:
            raise ValueError("dtype is bfloat16 or float16")
        self.state, self.dtype, self.device = state, dtype, state.device
        self.n_slots, self.Hv, self.Dk, self.Dv = state.shape
        self.Hk = Hk
        if Hk < 1 or self.Hv % Hk:
            raise ValueError("Hk must divide Hv")
        d = self.desc = moe_linear_desc()
        d.n_slots, d.Hk, d.Hv, d.Dk, d.Dv = self.n_slots, Hk, self.Hv, self.Dk, self.Dv
        d.dtype, d.state = _DTYPES[dtype], state.data_ptr()
        self._desc_ref = ctypes.byref(d)
        self._status = torch.zeros(1, dtype=_I32, device=self.device)
        self._status_ptr = self._status.data_ptr()

    def _heads(self, t, heads, D, what):
        """-> row stride of [rows][heads][D] with contiguous heads."""
        shape = t.shape
        if len(shape) != 3 or shape[1] != heads or shape[2] != D or t.dtype != self.dtype or t.device != self.device:
            raise ValueError(f"{what} must be [rows][{heads}][{D}] {self.dtype} on {self.device}")
        s0, s1, s2 = t.stride()
        if (s2 != 1 and D > 1) or (s1 != D and heads > 1):
            raise ValueError(f"{what}: the heads of a row must be contiguous")
        return s0 if shape[0] > 1 else heads * D  # (the distance to a next row says nothing of one)

    def _ints(self, t, what):
        if t.dtype != _I32 or t.device != self.device or not t.is_contiguous():
            raise ValueError(f"{what} must be a contiguous int32 tensor on {self.device}")
        return t

    def _call(self, fn, q, k, v, g, slots, row_start, scale, out, stream):
        q_stride, k_stride = self._heads(q, self.Hk, self.Dk, "q"), self._heads(k, self.Hk, self.Dk, "k")
        v_stride = self._heads(v, self.Hv, self.Dv, "v")
        n = q.shape[0]
        if k.shape[0] != n or v.shape[0] != n or n >= 1 << 31:
            raise ValueError("q, k and v must have the same rows, fewer than 2^31")
        shape, strides = g.shape, g.stride()
        if g.dtype != _F32 or g.device != self.device or shape not in ((n, self.Hv), (self.Hv,)) or \
                (strides[-1] != 1 and self.Hv > 1):
            raise ValueError(f"g must be fp32 [{n}][{self.Hv}] or [{self.Hv}] on {self.device}, heads contiguous")
        g_stride = 0 if len(shape) == 1 else strides[0] if n > 1 else self.Hv
        B = n if slots is None else self._ints(slots, "slots").numel()
        if row_start is not None:
            m = self._ints(row_start, "row_start").numel() - 1
            if m < 0 or (slots is not None and B != m):
                raise ValueError("row_start has one entry more than there are sequences")
            B = m
        if (n > 0 and B < 1) or (slots is None and B > self.n_slots):
            raise ValueError("more sequences than slots, or none")
        handle = _on(self.device, stream)
        if out is None:
            out = _new((n, self.Hv, self.Dv), self.dtype, self.device, stream)
        elif out.shape != v.shape or out.dtype != self.dtype or not out.is_contiguous() or out.device != self.device:
            raise ValueError("out must be a contiguous tensor like v")
        r = moe_kv_rows(B, n, None if slots is None else slots.data_ptr(), None if row_start is None else row_start.data_ptr())
        a = moe_linear_args(q.data_ptr(), k.data_ptr(), v.data_ptr(), q_stride, k_stride, v_stride, g.data_ptr(), g_stride,
                            self.Dk ** -0.5 if scale is None else scale, out.data_ptr(), self._status_ptr)
        fn(self._desc_ref, ctypes.byref(r), ctypes.byref(a), handle)
        return out

    def step(self, q, k, v, g, slots=None, scale=None, out=None, stream=None):
        """A decode window: the same number of rows (up to 16) for each slot (slots None: a
        row for each of the first slots). q, k [rows][Hk][Dk], v [rows][Hv][Dv]; g, the
        logarithms of the decays, fp32 [rows][Hv], or [Hv] for all rows; scale Dk^-0.5
        unless given. -> o [rows][Hv][Dv]."""
        return self._call(_lib.moe_linear_step, q, k, v, g, slots, None, scale, out, stream)

    def chunk(self, q, k, v, g, slots=None, row_start=None, scale=None, out=None, stream=None):
        """Prompt chunks: rows row_start[b] .. row_start[b + 1) belong to slot slots[b]
        (row_start None: the same number each). Sequences of one row or a few are better
        off in a call of step."""
        return self._call(_lib.moe_linear_chunk, q, k, v, g, slots, row_start, scale, out, stream)

    def status(self, stream=None):
        """-> device status bits: 2 a slot out of range, 64 a slot twice in a call, 4 a bounded
        wait of a chunk expired (its results are incomplete); waits."""
        handle = _on(self.device, stream)
        torch.cuda.ExternalStream(handle).synchronize() if handle else torch.cuda.default_stream().synchronize()
        return int(self._status)

    def clear_status(self, stream=None):
        with _lib.on_stream(stream):
            self._status.zero_()

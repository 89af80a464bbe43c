"""A paged key-value cache and its attention (include/moe_kv.h) over torch tensors.

`PagedKV` holds the pools, the page tables and the free stack of one model's
cache (or wraps a program's own tensors, `PagedKV.over`) with a workspace, and
forwards calls to libmoe_gb300.so: growing, forking, freeing and compacting
slots, writing new tokens' keys and values, and attention of decode windows and
prompt chunks. Marshalling only: tables, lengths and page numbers stay on the
GPU and no call waits for it, except `status()`.

A decode step of one sequence per slot, layer by layer:

    kv.grow(slots, ones)                     # pages for the new tokens
    for layer in range(n_layers):
        kv.append(layer, k, v, slots=slots)  # [B][Hkv][D] each
        o = kv.decode(layer, q, slots=slots) # [B][Hq][D]
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import _lib
from ._lib import MOE_KV_BF16, MOE_KV_F16, moe_attn_args, moe_kv_desc, moe_kv_rows

_DTYPES = {torch.bfloat16: MOE_KV_BF16, torch.float16: MOE_KV_F16}
_I32, _F32 = torch.int32, torch.float32
# The current stream's handle without the Stream object around it: a decode step
# makes two calls per layer, and the object costs as much as a launch.
_current_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice


def _i32(t, what, device):
    if t.dtype != _I32 or t.device != device or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous int32 tensor on {device}")
    return t


class PagedKV:
    """k, v [n_layers][n_pages][Hkv][page_size][D] (bf16 or fp16), table int32
    [n_slots][max_pages], lens int32 [n_slots], refs int32 [n_pages], free int32
    [n_pages] with n_free int32 [1]. Hq: query heads; max_rows: rows of the
    largest decode call (sizes the workspace; chunks may have more). One thread at a time: the
    calls share the argument structs and the workspace. A call works on the
    current stream, or on `stream` (a torch stream or a handle), whose the results
    are then; ordering it with other streams, and keeping the arguments alive until
    it has run, is the caller's."""

    def __init__(self, n_layers, n_pages, page_size, Hkv, D, n_slots, max_pages, Hq=None, max_rows=2048,
                 dtype=torch.bfloat16, device="cuda"):
        i32 = dict(dtype=torch.int32, device=device)
        k = torch.zeros(n_layers, n_pages, Hkv, page_size, D, dtype=dtype, device=device)
        self._setup(k, torch.zeros_like(k), torch.full((n_slots, max_pages), -1, **i32), torch.zeros(n_slots, **i32),
                    torch.zeros(n_pages, **i32), torch.arange(n_pages - 1, -1, -1, **i32),
                    torch.full((1,), n_pages, **i32), Hkv if Hq is None else Hq, max_rows)

    @classmethod
    def over(cls, k, v, table, lens, refs, free, n_free, Hq=None, max_rows=2048):
        """A cache over the caller's tensors (used in place)."""
        self = cls.__new__(cls)
        self._setup(k, v, table, lens, refs, free, n_free, k.shape[2] if Hq is None else Hq, max_rows)
        return self

    def _setup(self, k, v, table, lens, refs, free, n_free, Hq, max_rows):
        if k.dim() != 5 or k.dtype not in _DTYPES or not k.is_contiguous():
            raise ValueError("k must be a contiguous bf16 or fp16 [n_layers][n_pages][Hkv][page_size][D]")
        if v.shape != k.shape or v.dtype != k.dtype or not v.is_contiguous() or v.device != k.device:
            raise ValueError("v must be like k")
        dev = k.device
        n_layers, n_pages, Hkv, page, D = k.shape
        if table.dim() != 2 or lens.numel() != table.shape[0] or refs.numel() != n_pages or \
                free.numel() != n_pages or n_free.numel() != 1:
            raise ValueError("table [n_slots][max_pages], lens [n_slots], refs and free [n_pages], n_free [1]")
        for t, what in ((table, "table"), (lens, "lens"), (refs, "refs"), (free, "free"), (n_free, "n_free")):
            _i32(t, what, dev)
        self.k, self.v, self.table, self.lens, self.refs, self.free, self.n_free = k, v, table, lens, refs, free, n_free
        self.Hkv, self.D, self.Hq, self.device, self.dtype = Hkv, D, Hq, dev, k.dtype
        d = self.desc = moe_kv_desc()
        d.k, d.v, d.dtype = k.data_ptr(), v.data_ptr(), _DTYPES[k.dtype]
        d.n_layers, d.n_pages, d.page_size, d.Hkv, d.D = n_layers, n_pages, page, Hkv, D
        d.n_slots, d.max_pages = table.shape
        d.table, d.lens, d.refs = table.data_ptr(), lens.data_ptr(), refs.data_ptr()
        d.free_pages, d.n_free = free.data_ptr(), n_free.data_ptr()
        self.n_slots, self.max_rows = d.n_slots, max_rows
        self.ws_bytes = _lib.moe_kv_workspace_bytes(d, Hq, max_rows)
        if self.ws_bytes == 0:
            raise ValueError("unsupported cache: see moe_kv_desc for the limits")
        self._index = dev.index or 0
        if dev.type == "cuda":
            self._stream(None)
        self.ws = torch.empty(self.ws_bytes + 256, dtype=torch.uint8, device=dev)
        self.ws_ptr = self.ws.data_ptr() + (-self.ws.data_ptr()) % 256
        _lib.moe_workspace_init(self.ws_ptr, self.ws_bytes)
        self._desc_ref = ctypes.byref(d)
        self._rows, self._args = moe_kv_rows(), moe_attn_args()
        self._rows_ref, self._args_ref = ctypes.byref(self._rows), ctypes.byref(self._args)
        self._args.Hq, self._scale = Hq, 1.0 / math.sqrt(D)

    # ---- marshalling
    def _stream(self, stream):
        if _current_device() != self._index:  # the library launches on the current device
            raise ValueError(f"the cache is on {self.device}, the current device is cuda:{_current_device()}")
        if stream is None:
            return _current_stream(self._index)
        return stream if isinstance(stream, int) else stream.cuda_stream

    def _new(self, shape, dtype, stream):
        if stream is None:
            return torch.empty(shape, dtype=dtype, device=self.device)
        with _lib.on_stream(stream):
            return torch.empty(shape, dtype=dtype, device=self.device)

    def _heads(self, t, heads, what):
        """-> row stride of [rows][heads][D] with contiguous heads."""
        shape, D = t.shape, self.D
        if len(shape) != 3 or shape[1] != heads or shape[2] != D or t.dtype != self.dtype or t.device != self.device:
            raise ValueError(f"{what} must be [rows][{heads}][{D}] {self.dtype} on {self.device}")
        s0, s1, s2 = t.stride()
        if s2 != 1 or (s1 != D and heads > 1):
            raise ValueError(f"{what}: the heads of a row must be contiguous")
        return s0 if shape[0] > 1 else heads * D  # (the distance to a next row says nothing of one)

    def _set_rows(self, n_rows, slots, row_start):
        r = self._rows
        if slots is None:
            B, r.slots = n_rows, None
        else:
            B, r.slots = _i32(slots, "slots", self.device).numel(), slots.data_ptr()
        if row_start is None:
            r.row_start = None
        else:
            n = _i32(row_start, "row_start", self.device).numel() - 1
            if n < 0 or (slots is not None and B != n):
                raise ValueError("row_start has one entry more than there are sequences")
            B, r.row_start = n, row_start.data_ptr()
        if (n_rows > 0 and B < 1) or (slots is None and B > self.n_slots):
            raise ValueError("more sequences than slots, or none")
        r.B, r.n_rows = B, n_rows

    # ---- new tokens and attention
    def append(self, layer, k, v, slots=None, row_start=None, stream=None):
        """Write k, v [rows][Hkv][D] of the newest tokens into `layer`'s pages."""
        stride = self._heads(k, self.Hkv, "k")
        n = k.shape[0]
        if self._heads(v, self.Hkv, "v") != stride or v.shape[0] != n:
            raise ValueError("k and v must have the same rows and row stride")
        self._set_rows(n, slots, row_start)
        _lib.moe_kv_append(self._desc_ref, layer, self._rows_ref, k.data_ptr(), v.data_ptr(), stride, self.ws_ptr,
                           self.ws_bytes, self._stream(stream))

    def append_rotary(self, layer, q, k, v, rotary, slots=None, row_start=None, positions=None, q_out=None, stream=None):
        """append with rotary positions: the rows' keys are turned on their way into the
        pages, their queries q [rows][Hq][D] into q_out (a new tensor unless given; may
        be q). rotary: a `block.Rotary`; positions int32 [rows] (None: each row's token
        number in its sequence). -> q_out."""
        Hq = self.Hq
        q_stride, stride = self._heads(q, Hq, "q"), self._heads(k, self.Hkv, "k")
        n = q.shape[0]
        if self._heads(v, self.Hkv, "v") != stride or k.shape[0] != n or v.shape[0] != n:
            raise ValueError("q, k and v must have the same rows, k and v the same row stride")
        if rotary.device != self.device:
            raise ValueError(f"the rotary frequencies are on {rotary.device}, the cache on {self.device}")
        if positions is not None and _i32(positions, "positions", self.device).numel() != n:
            raise ValueError("one position per row")
        self._set_rows(n, slots, row_start)
        if q_out is None:
            q_out = self._new((n, Hq, self.D), self.dtype, stream)
        elif q_out.shape != q.shape:
            raise ValueError("q_out must be like q")
        _lib.moe_kv_append_rope(self._desc_ref, layer, self._rows_ref, rotary.desc_ref,
                                None if positions is None else positions.data_ptr(), Hq, q.data_ptr(), q_stride,
                                q_out.data_ptr(), self._heads(q_out, Hq, "q_out"), k.data_ptr(), v.data_ptr(), stride,
                                self.ws_ptr, self.ws_bytes, self._stream(stream))
        return q_out

    def _attend(self, fn, layer, q, slots, row_start, scale, window, sinks, want_lse, out, lse, stream):
        Hq = self.Hq
        stride = self._heads(q, Hq, "q")
        n = q.shape[0]
        self._set_rows(n, slots, row_start)
        if out is None:
            out = self._new((n, Hq, self.D), self.dtype, stream)
        elif out.shape != q.shape or out.dtype != self.dtype or not out.is_contiguous() or out.device != self.device:
            raise ValueError("out must be a contiguous tensor like q")
        if lse is None:
            if want_lse:
                lse = self._new((n, Hq), _F32, stream)
        elif lse.shape != (n, Hq) or lse.dtype != _F32 or not lse.is_contiguous() or lse.device != self.device:
            raise ValueError("lse must be a contiguous fp32 [rows][Hq]")
        a = self._args
        a.scale, a.window, a.n_sink = (self._scale if scale is None else scale), window, sinks
        a.q, a.q_stride, a.o = q.data_ptr(), stride, out.data_ptr()
        a.lse = None if lse is None else lse.data_ptr()
        fn(self._desc_ref, layer, self._rows_ref, self._args_ref, self.ws_ptr, self.ws_bytes, self._stream(stream))
        return out if lse is None else (out, lse)

    def decode(self, layer, q, slots=None, scale=None, window=0, sinks=0, want_lse=False, out=None, lse=None,
               stream=None):
        """Attention of a decode window: q [rows][Hq][D], the same number of rows
        (up to 16) for each slot (slots None: a row for each of the first slots).
        -> o, or (o, lse) with want_lse."""
        if q.dim() == 3 and q.shape[0] > self.max_rows:
            raise ValueError(f"{q.shape[0]} rows: the workspace is sized for {self.max_rows}")
        return self._attend(_lib.moe_attn_decode, layer, q, slots, None, scale, window, sinks, want_lse, out, lse, stream)

    def chunk(self, layer, q, slots=None, row_start=None, scale=None, window=0, sinks=0, want_lse=False, out=None,
              lse=None, stream=None):
        """Attention of prompt chunks: rows row_start[b] .. row_start[b + 1) of q
        belong to slot slots[b] (row_start None: the same number each)."""
        return self._attend(_lib.moe_attn_chunk, layer, q, slots, row_start, scale, window, sinks, want_lse, out, lse,
                            stream)

    # ---- pages
    def grow(self, slots, add, stream=None):
        """Pages for add[i] more tokens of slot slots[i]."""
        _i32(slots, "slots", self.device), _i32(add, "add", self.device)
        if add.numel() != slots.numel():
            raise ValueError("one add per slot")
        _lib.moe_kv_grow(self._desc_ref, slots.data_ptr(), add.data_ptr(), slots.numel(), self.ws_ptr, self.ws_bytes, self._stream(stream))

    def fork(self, src, dst, stream=None):
        """Slot dst[i] (empty) becomes a fork of slot src[i]."""
        _i32(src, "src", self.device), _i32(dst, "dst", self.device)
        if src.numel() != dst.numel():
            raise ValueError("one dst per src")
        _lib.moe_kv_fork(self._desc_ref, src.data_ptr(), dst.data_ptr(), src.numel(), self.ws_ptr, self.ws_bytes, self._stream(stream))

    def free_slots(self, slots, stream=None):
        """Empty the slots; pages that no slot holds any more become free."""
        _i32(slots, "slots", self.device)
        _lib.moe_kv_free(self._desc_ref, slots.data_ptr(), slots.numel(), self.ws_ptr, self.ws_bytes, self._stream(stream))

    def compact(self, n_moved=None, stream=None):
        """Move the live pages to the lowest page numbers (n_moved: int32 [1], the moves)."""
        if n_moved is not None:
            _i32(n_moved, "n_moved", self.device)
        _lib.moe_kv_compact(self._desc_ref, n_moved, self.ws_ptr, self.ws_bytes, self._stream(stream))

    def copy_pages(self, src, dst, stream=None):
        """Copy page src[i] to page dst[i] in every layer."""
        _i32(src, "src", self.device), _i32(dst, "dst", self.device)
        if src.numel() != dst.numel():
            raise ValueError("one dst per src")
        _lib.moe_kv_copy_pages(self._desc_ref, src.data_ptr(), dst.data_ptr(), src.numel(), self.ws_ptr, self.ws_bytes,
                               self._stream(stream))

    def status(self, stream=None):
        """-> (moe_status code, raw device status bits); waits for the stream."""
        return _lib.moe_read_status(self.ws_ptr, self._stream(stream))

    def clear_status(self, stream=None):
        _lib.moe_workspace_init(self.ws_ptr, self.ws_bytes, self._stream(stream))

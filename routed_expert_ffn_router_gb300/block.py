"""What a decoder layer has around its attention and its experts
(include/moe_block.h) over torch tensors: the norm with the residual's addition,
rotary positions for `PagedKV.append_rotary`, and log probabilities of tokens.

A layer of a decoder, with x the output of the one before:

    h = rms_norm(x, w1, residual=r)                        # r += x; h = norm(r) w1
    q, k, v = split(h @ wqkv)
    q = kv.append_rotary(l, q, k, v, rotary, slots=slots)  # into the pages
    x = kv.decode(l, q, slots=slots).flatten(1) @ wo
    h = rms_norm(x, w2, residual=r)
    x = moe.forward(h.float() @ router, h)["y"]            # joins r in the next norm

Marshalling only: the work is in libmoe_gb300.so. A call works on the current
stream of its tensors' device, which has to be the current one, or on `stream`
(a torch stream or a handle), to which new results then belong. Any number of
calls may be under way at once.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import _lib
from ._lib import MOE_ROPE_HALF, MOE_ROPE_INTERLEAVED, moe_logprobs_args, moe_norm_args, moe_rope_desc

_TYPES = {torch.float32: _lib.MOE_T_F32, torch.bfloat16: _lib.MOE_T_BF16, torch.float16: _lib.MOE_T_F16}
_E4M3 = torch.float8_e4m3fn
_OUT_TYPES = {**_TYPES, _E4M3: _lib.MOE_T_E4M3}
_I32, _F32 = torch.int32, torch.float32
_current_stream = torch._C._cuda_getCurrentRawStream


def _on(device, stream):
    """-> the stream's handle; the library launches on the current device."""
    now = torch._C._cuda_getDevice()
    if device.type != "cuda" or now != device.index:
        raise ValueError(f"the tensors are on {device}, the current device is cuda:{now}")
    if stream is None:
        return _current_stream(now)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _new(shape, dtype, device, stream):
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with _lib.on_stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _rows(t, shape, types, what, device):
    """-> (type, row stride) of a [T][H] tensor with contiguous rows."""
    kind = types.get(t.dtype)
    if kind is None or t.shape != shape or t.device != device:
        raise ValueError(f"{what} must be {list(shape)} on {device}, of {', '.join(str(x)[6:] for x in types)}")
    T, H = shape
    if T >= 1 << 31 or H >= 1 << 31:
        raise ValueError(f"{what}: more than 2^31 - 1 rows or columns")
    s0, s1 = t.stride()
    if s1 != 1 and H > 1:
        raise ValueError(f"{what}: the values of a row must be contiguous")
    if T <= 1:  # (the distance to a next row says nothing of one)
        return kind, H
    if s0 < H:
        raise ValueError(f"{what}: rows must not overlap")
    return kind, s0


def rms_norm(x, weight=None, residual=None, eps=1e-6, weight_offset=0.0, out_dtype=None, group=0, out=None, scales=None,
             stream=None):
    """residual += x (in place, rounded to its type), then the root-mean-square norm of
    the residual's rows (of x's without one) times weight + weight_offset.
    x, residual [rows][H] fp32, bf16 or fp16; weight [H]. -> y [rows][H] of out_dtype
    (the residual's type unless given) or out; with float8_e4m3fn (y, scales), y times
    scales [rows][H / group] being the norm (group 0: one scale per row; else a power
    of two from 16). out may be x."""
    shape, dev = x.shape, x.device
    if len(shape) != 2:
        raise ValueError("x must be [rows][H]")
    T, H = shape
    x_type, x_stride = _rows(x, shape, _TYPES, "x", dev)
    res_type = res_stride = w_type = 0
    res = w = s = None
    if residual is not None:
        res_type, res_stride = _rows(residual, shape, _TYPES, "residual", dev)
        res = residual.data_ptr()
    if weight is not None:
        w_type = _TYPES.get(weight.dtype)
        if w_type is None or weight.shape != (H,) or weight.device != dev or not weight.is_contiguous():
            raise ValueError(f"weight must be a contiguous [{H}] on {dev}, of fp32, bf16 or fp16")
        w = weight.data_ptr()
    handle = _on(dev, stream)
    if out is None:
        out = _new(shape, (x if residual is None else residual).dtype if out_dtype is None else out_dtype, dev, stream)
    elif out_dtype is not None and out.dtype != out_dtype:
        raise ValueError("out is not of out_dtype")
    y_type, y_stride = _rows(out, shape, _OUT_TYPES, "out", dev)
    if y_type != _lib.MOE_T_E4M3:
        if scales is not None or group:
            raise ValueError("scales and group are for float8_e4m3fn")
    else:
        if group < 0 or (group and H % group):
            raise ValueError("group must divide the row")
        n = H // group if group else 1
        if scales is None:
            scales = _new((T, n), _F32, dev, stream)
        elif scales.shape != (T, n) or scales.dtype != _F32 or not scales.is_contiguous() or scales.device != dev:
            raise ValueError(f"scales must be a contiguous fp32 [{T}][{n}] on {dev}")
        s = scales.data_ptr()
    _lib.moe_rms_norm(ctypes.byref(moe_norm_args(T, H, x_type, res_type, w_type, y_type, group, eps, weight_offset, x.data_ptr(),
                                                 x_stride, res, res_stride, w, out.data_ptr(), y_stride, s)), handle)
    return out if s is None else (out, scales)


_LOGPROB_OUT = (("logprob", _F32), ("rank", _I32), ("entropy", _F32), ("top_ids", _I32), ("top_logprobs", _F32))


def token_logprobs(logits, tokens=None, top=0, temperature=1.0, out=None, stream=None):
    """Log probabilities over logits [rows][V] (fp32, bf16 or fp16; any row stride) at a
    temperature. -> dict: entropy [rows]; with tokens (int32 [rows]) logprob and rank
    (0: the most likely one; a token outside [0, V): 0 and -1); with top (up to 32)
    top_ids and top_logprobs [rows][top], the most likely tokens in order, ties to the
    lower id. out: a dict of such tensors to write to."""
    shape, dev = logits.shape, logits.device
    if len(shape) != 2:
        raise ValueError("logits must be [rows][V]")
    T, V = shape
    kind, stride = _rows(logits, shape, _TYPES, "logits", dev)
    if tokens is not None and (tokens.shape != (T,) or tokens.dtype != _I32 or not tokens.is_contiguous() or tokens.device != dev):
        raise ValueError(f"tokens must be a contiguous int32 [{T}] on {dev}")
    if top < 0:
        raise ValueError("top must not be negative")
    handle = _on(dev, stream)
    r, at = {}, []
    for name, dtype in _LOGPROB_OUT:
        wide = name[0] == "t"
        if (not top) if wide else (tokens is None and name != "entropy"):
            at.append(None)
            continue
        want = (T, top) if wide else (T,)
        if out is None:
            t = _new(want, dtype, dev, stream)
        else:
            t = out.get(name)
            if t is None or t.shape != want or t.dtype != dtype or not t.is_contiguous() or t.device != dev:
                raise ValueError(f"out[{name!r}] must be a contiguous {str(dtype)[6:]} {list(want)} on {dev}")
        r[name] = t
        at.append(t.data_ptr())
    _lib.moe_token_logprobs(ctypes.byref(moe_logprobs_args(T, V, top, kind, temperature, logits.data_ptr(), stride,
                                                           None if tokens is None else tokens.data_ptr(), *at)), handle)
    return r


def rotary_frequencies(rot, base=10000.0, scaling=None):
    """-> (radians per token of each of the rot / 2 pairs, gain). scaling: None or a dict:
      kind "linear": factor           positions divided by it;
      kind "ntk":    factor           base times factor^(rot / (rot - 2));
      kind "yarn":   factor, original [, fast = 32, slow = 1, gain]
        pairs that turn more than `fast` times in the original context keep their
        frequency, those below `slow` turns have it divided, a ramp over the pairs
        between; gain 0.1 ln(factor) + 1 (Peng et al., 2023);
      kind "bands":  factor, original, low, high
        the same by wavelengths: original / wavelength above `high` keeps, below `low`
        is divided, linear between."""
    f = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if scaling is None:
        return f, 1.0
    s = dict(scaling)
    kind, factor = s.pop("kind"), float(s.pop("factor"))
    gain = 1.0
    if not factor > 0:
        raise ValueError("factor must be above 0")
    if kind == "linear":
        f = [x / factor for x in f]
    elif kind == "ntk":
        if rot > 2:
            f = [(base * factor ** (rot / (rot - 2.0))) ** (-2.0 * i / rot) for i in range(rot // 2)]
    elif kind == "yarn":
        original, fast, slow = float(s.pop("original")), float(s.pop("fast", 32.0)), float(s.pop("slow", 1.0))
        gain = float(s.pop("gain", 0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0))

        def pair(turns):  # the (fractional) pair that turns so often
            return rot * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo, hi = max(math.floor(pair(fast)), 0), min(math.ceil(pair(slow)), rot - 1)
        ramp = [min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0) for i in range(rot // 2)]
        f = [x * (1 - r) + x / factor * r for x, r in zip(f, ramp)]
    elif kind == "bands":
        original, low, high = float(s.pop("original")), float(s.pop("low")), float(s.pop("high"))
        if not high > low:
            raise ValueError("high must be above low")
        keep = [min(max((original * x / (2 * math.pi) - low) / (high - low), 0.0), 1.0) for x in f]
        f = [x * k + x / factor * (1 - k) for x, k in zip(f, keep)]
    else:
        raise ValueError(f"no scaling of kind {kind!r}")
    if s:
        raise ValueError(f"scaling {kind!r} has no {', '.join(sorted(s))}")
    return f, gain


class Rotary:
    """Rotary positions of a head's first `rot` values: layout "half" pairs (i, i + rot
    / 2), "interleaved" (2 i, 2 i + 1). Frequencies from base and scaling
    (`rotary_frequencies`), or given: radians per token of each pair, with a gain."""

    def __init__(self, rot, base=10000.0, layout="half", scaling=None, frequencies=None, gain=None, device="cuda"):
        if rot < 2 or rot % 2:
            raise ValueError("rot must be even, from 2")
        if layout not in ("half", "interleaved"):
            raise ValueError("layout is half or interleaved")
        if frequencies is None:
            frequencies, own_gain = rotary_frequencies(rot, base, scaling)
        elif len(frequencies) != rot // 2 or scaling is not None:
            raise ValueError("one frequency per pair, without a scaling")
        else:
            own_gain = 1.0
        self.rot, self.layout, self.frequencies = rot, layout, [float(x) for x in frequencies]
        self.gain = float(own_gain if gain is None else gain)
        turns = [round(x / (2 * math.pi) * 2.0 ** 64) % 2 ** 64 for x in self.frequencies]
        device = torch.device(device)
        if device.type == "cuda" and device.index is None:
            device = torch.device("cuda", torch._C._cuda_getDevice())
        # as int64: the same bits
        self.freq = torch.tensor([x - 2 ** 64 if x >= 2 ** 63 else x for x in turns], dtype=torch.int64, device=device)
        self.device = device
        d = self.desc = moe_rope_desc()
        d.rot, d.gain, d.freq = rot, self.gain, self.freq.data_ptr()
        d.layout = MOE_ROPE_HALF if layout == "half" else MOE_ROPE_INTERLEAVED
        self.desc_ref = ctypes.byref(d)

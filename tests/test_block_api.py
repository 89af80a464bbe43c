"""The decoder-block C ABI (include/moe_block.h, moe_kv_append_rope) refuses bad
arguments on the host before anything is launched, and its Python wrappers check
what they marshal. No GPU needed."""
import ctypes
import math
import os
import re

import pytest
import torch

from routed_expert_ffn_router_gb300 import _lib, block
from routed_expert_ffn_router_gb300 import build as libbuild
from routed_expert_ffn_router_gb300.block import Rotary, rms_norm, rotary_frequencies, token_logprobs
from routed_expert_ffn_router_gb300.linear import LinearAttention
from tests._kv_ref import Case
from tests.test_kv_api import desc, rows

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INV, UNS, WS, OK = _lib.MOE_ERR_INVALID, _lib.MOE_ERR_UNSUPPORTED, _lib.MOE_ERR_WORKSPACE, _lib.MOE_OK
A, B = 4096, 1 << 20  # aligned addresses that nothing touches


@pytest.fixture(scope="module", autouse=True)
def lib():
    libbuild.build()
    return _lib.load()


def test_every_declared_symbol_is_exported(lib):
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "moe_block.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(moe_[a-z_]+)\s*\(", src))
    assert names == set(_lib.BLOCK_EXPORTS) and all(hasattr(lib, n) for n in names)


def struct(cls, **kw):
    s = cls()
    for n, x in kw.items():
        setattr(s, n, x)
    return s


NORM = dict(T=4, H=256, x_type=1, res_type=1, w_type=1, y_type=1, eps=1e-6, x=A, x_stride=256, res=B, res_stride=256, w=A, y=2 * B,
            y_stride=256)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), INV), (dict(H=0), INV), (dict(H=16385, x_stride=20000, y_stride=20000, res_stride=20000), UNS), (dict(x=None), INV),
    (dict(y=None), INV), (dict(x_type=3), INV), (dict(res_type=3), INV), (dict(w_type=5), INV), (dict(y_type=4), INV),
    (dict(y_type=-1), INV), (dict(eps=-1.0), INV), (dict(eps=math.nan), INV), (dict(w_offset=math.inf), INV),
    (dict(x_stride=255), INV), (dict(res_stride=255), INV), (dict(y_stride=255), INV), (dict(group=32), INV),
    (dict(y_type=3), INV), (dict(y_type=3, scales=A, group=24), INV), (dict(y_type=3, scales=A, group=8), INV),
    (dict(y_type=3, scales=A, group=512), INV), (dict(y_type=3, scales=A + 2), INV), (dict(x=A + 1), INV), (dict(res=B + 1), INV),
    (dict(w=A + 1), INV), (dict(x_type=0, x=A + 2), INV), (dict(res=A), INV), (dict(y=B), INV), (dict(y=A, y_type=2), INV),
    (dict(y=A, y_stride=264), INV), (dict(T=0, x=None, y=None), OK),
])
def test_norm_refusals(lib, kw, code):
    assert lib.moe_rms_norm(ctypes.byref(struct(_lib.moe_norm_args, **{**NORM, **kw})), None) == code
    assert lib.moe_rms_norm(None, None) == INV


LOGP = dict(T=2, V=100, top=4, type=1, temperature=1.0, logits=A, stride=100, tokens=A, logprob=A, rank=A, entropy=A, top_ids=A,
            top_logprobs=A)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), INV), (dict(V=0), INV), (dict(top=-1), INV), (dict(type=3), INV), (dict(temperature=0.0), INV),
    (dict(temperature=-1.0), INV), (dict(temperature=math.nan), INV), (dict(temperature=math.inf), INV),
    (dict(temperature=1e-38), INV), (dict(top=33), UNS), (dict(V=3, top=4), UNS), (dict(V=1 << 29, stride=1 << 29), UNS),
    (dict(logits=None), INV), (dict(logits=A + 1), INV), (dict(type=0, logits=A + 2), INV), (dict(stride=99), INV),
    (dict(tokens=None), INV), (dict(top_ids=None), INV), (dict(top_logprobs=None), INV), (dict(top=0), INV),
    (dict(logprob=A + 2), INV), (dict(top_ids=A + 1), INV), (dict(T=0, logits=None), OK),
])
def test_logprobs_refusals(lib, kw, code):
    assert lib.moe_token_logprobs(ctypes.byref(struct(_lib.moe_logprobs_args, **{**LOGP, **kw})), None) == code
    assert lib.moe_token_logprobs(None, None) == INV


LDESC = dict(n_slots=8, Hk=2, Hv=4, Dk=128, Dv=128, dtype=1, state=A)
LARGS = dict(q=A, k=A, v=A, q_stride=1024, k_stride=1024, v_stride=1024, g=A, g_stride=4, scale=1.0, o=A, status=A)


@pytest.mark.parametrize("d,a,r,code", [
    (dict(n_slots=0), {}, {}, INV), (dict(Hk=0), {}, {}, INV), (dict(Hv=5), {}, {}, INV), (dict(Hv=0), {}, {}, INV),
    (dict(Dk=0), {}, {}, INV), (dict(Dk=12), {}, {}, UNS), (dict(Dv=264), {}, {}, UNS), (dict(Hv=65536), {}, {}, UNS),
    (dict(n_slots=1 << 21), {}, {}, UNS), (dict(dtype=0), {}, {}, INV), (dict(dtype=3), {}, {}, INV), (dict(state=None), {}, {}, INV),
    (dict(state=A + 4), {}, {}, INV), ({}, dict(q=None), {}, INV), ({}, dict(k=A + 8), {}, INV), ({}, dict(v=None), {}, INV),
    ({}, dict(g=None), {}, INV), ({}, dict(g=A + 2), {}, INV), ({}, dict(o=A + 2), {}, INV), ({}, dict(q_stride=255), {}, INV),
    ({}, dict(q_stride=260), {}, INV), ({}, dict(v_stride=504), {}, INV), ({}, dict(g_stride=3), {}, INV),
    ({}, dict(g_stride=-1), {}, INV), ({}, dict(scale=math.nan), {}, INV), ({}, dict(status=A + 1), {}, INV),
    ({}, {}, dict(B=-1), INV), ({}, {}, dict(n_rows=-1), INV), ({}, {}, dict(B=0), INV), ({}, {}, dict(n_rows=5), INV),
    ({}, {}, dict(slots=A + 1), INV), ({}, dict(q=None), dict(n_rows=0), OK),
])
def test_linear_refusals(lib, d, a, r, code):
    d, a = struct(_lib.moe_linear_desc, **{**LDESC, **d}), struct(_lib.moe_linear_args, **{**LARGS, **a})
    for fn in (lib.moe_linear_step, lib.moe_linear_chunk):
        assert fn(ctypes.byref(d), ctypes.byref(rows(**r)), ctypes.byref(a), None) == code
        assert fn(None, ctypes.byref(rows()), ctypes.byref(a), None) == INV
        assert fn(ctypes.byref(d), None, ctypes.byref(a), None) == INV
        assert fn(ctypes.byref(d), ctypes.byref(rows()), None, None) == INV


def test_step_takes_equal_rows_of_at_most_16(lib):
    d, a = struct(_lib.moe_linear_desc, **LDESC), struct(_lib.moe_linear_args, **LARGS)
    f = lambda **kw: lib.moe_linear_step(ctypes.byref(d), ctypes.byref(rows(**kw)), ctypes.byref(a), None)  # noqa: E731
    assert f(row_start=A) == INV and f(B=2, n_rows=34) == UNS
    big = struct(_lib.moe_linear_desc, **{**LDESC, "Hv": 65534})
    assert lib.moe_linear_step(ctypes.byref(big), ctypes.byref(rows(B=1 << 16, n_rows=1 << 16)), ctypes.byref(a), None) == UNS


def rope(**kw):
    return struct(_lib.moe_rope_desc, **{**dict(rot=128, layout=0, gain=1.0, freq=A), **kw})


@pytest.mark.parametrize("ro,kw,code", [
    (dict(rot=0), {}, INV), (dict(rot=3), {}, INV), (dict(rot=130), {}, INV), (dict(layout=2), {}, INV), (dict(gain=math.nan), {}, INV),
    (dict(freq=None), {}, INV), (dict(freq=A + 4), {}, INV), ({}, dict(Hq=0), INV), ({}, dict(Hq=65536, q_stride=1 << 24), UNS),
    ({}, dict(q=None), INV), ({}, dict(q_out=None), INV), ({}, dict(q=A + 8), INV), ({}, dict(q_out=A + 2), INV),
    ({}, dict(q_stride=16 * 128 - 8), INV), ({}, dict(q_stride=16 * 128 + 4), INV), ({}, dict(q_out_stride=8), INV),
    ({}, dict(q_out=A, q_out_stride=16 * 128 + 8), INV), ({}, dict(k=None), INV), ({}, dict(v=A + 8), INV),
    ({}, dict(row_stride=4 * 128 - 8), INV), ({}, dict(positions=A + 2), INV), ({}, dict(ws=A + 16), WS), ({}, dict(ws_bytes=64), WS),
])
def test_rope_refusals(lib, ro, kw, code):
    a = {**dict(positions=None, Hq=16, q=A, q_stride=16 * 128, q_out=B, q_out_stride=16 * 128, k=A, v=A, row_stride=4 * 128, ws=A,
                ws_bytes=1 << 40), **kw}
    call = lambda d, r, ro: lib.moe_kv_append_rope(d, 0, r, ro, a["positions"], a["Hq"], a["q"], a["q_stride"], a["q_out"],  # noqa: E731
                                                   a["q_out_stride"], a["k"], a["v"], a["row_stride"], a["ws"], a["ws_bytes"], None)
    assert call(ctypes.byref(desc()), ctypes.byref(rows()), ctypes.byref(rope(**ro))) == code
    assert call(ctypes.byref(desc()), ctypes.byref(rows()), None) == INV
    assert call(None, ctypes.byref(rows()), ctypes.byref(rope())) == INV
    assert call(ctypes.byref(desc(D=100)), ctypes.byref(rows()), ctypes.byref(rope(rot=64))) == UNS


# ------------------------------------------------------------------ frequencies
def test_frequencies():
    f, gain = rotary_frequencies(8)
    assert gain == 1 and f == pytest.approx([1, 0.1, 0.01, 0.001])
    assert rotary_frequencies(8, scaling=dict(kind="linear", factor=4))[0] == pytest.approx([x / 4 for x in f])
    # ntk: the first pair keeps its frequency, the last is divided by the factor
    n = rotary_frequencies(8, scaling=dict(kind="ntk", factor=4))[0]
    assert n[0] == 1 and n[-1] == pytest.approx(f[-1] / 4)
    f = rotary_frequencies(128)[0]
    y, gain = rotary_frequencies(128, scaling=dict(kind="yarn", factor=4, original=8192))
    assert gain == pytest.approx(1 + 0.1 * math.log(4))
    turns = [8192 * x / (2 * math.pi) for x in f]
    assert all(a == b for a, b, t in zip(y, f, turns) if t > 40)
    assert all(a == pytest.approx(b / 4) for a, b, t in zip(y, f, turns) if t < 0.8)
    assert all(b / 4 <= a * (1 + 1e-12) and a <= b for a, b in zip(y, f))
    b = rotary_frequencies(128, scaling=dict(kind="bands", factor=8, original=8192, low=1, high=4))[0]
    assert all(x == pytest.approx(z if t > 4 else z / 8) for x, z, t in zip(b, f, turns) if t > 4 or t < 1)
    mid = [(x, z, t) for x, z, t in zip(b, f, turns) if 1 <= t <= 4]
    assert mid and all(x == pytest.approx(z / 8 + (z - z / 8) * (t - 1) / 3) for x, z, t in mid)
    for bad in (dict(kind="other", factor=2), dict(kind="linear", factor=0), dict(kind="linear", factor=2, low=1),
                dict(kind="bands", factor=2, original=8, low=4, high=4)):
        with pytest.raises(ValueError):
            rotary_frequencies(64, scaling=bad)


def test_rotary_holds_turns_of_2_64():
    r = Rotary(4, frequencies=[2 * math.pi * 0.75, 2 * math.pi / 1024], device="cpu")
    assert [x % 2 ** 64 for x in r.freq.tolist()] == [3 * 2 ** 62, 2 ** 54] and r.gain == 1
    # far positions: p times the fraction, modulo a turn, against exact rationals
    r = Rotary(128, device="cpu")
    for f, x in zip(r.freq.tolist(), r.frequencies):
        p = 1_000_003
        got = (f % 2 ** 64) * p % 2 ** 64 / 2 ** 64
        want = p * x / (2 * math.pi) % 1.0
        assert min(abs(got - want), 1 - abs(got - want)) < 1e-9
    for kw in (dict(rot=3), dict(rot=0), dict(rot=4, layout="x"), dict(rot=4, frequencies=[1.0]),
               dict(rot=4, frequencies=[1.0, 1.0], scaling=dict(kind="linear", factor=2))):
        with pytest.raises(ValueError):
            Rotary(device="cpu", **kw)


# ------------------------------------------------------------------ wrappers
@pytest.fixture
def calls(monkeypatch):
    got = []
    for n in ("moe_rms_norm", "moe_token_logprobs", "moe_linear_step", "moe_linear_chunk", "moe_kv_append_rope"):
        monkeypatch.setattr(_lib, n, lambda *a, n=n: got.append(n))
    monkeypatch.setattr(block, "_on", lambda device, stream: 0)
    from routed_expert_ffn_router_gb300 import linear
    monkeypatch.setattr(linear, "_on", lambda device, stream: 0)
    return got


def test_norm_wrapper(calls):
    x, w = torch.zeros(3, 64), torch.zeros(64)
    E4 = torch.float8_e4m3fn
    assert rms_norm(x, w).shape == (3, 64) and rms_norm(x, residual=x.bfloat16()).dtype == torch.bfloat16
    q, s = rms_norm(x, out_dtype=E4, group=16)
    assert q.dtype == E4 and s.shape == (3, 4)
    assert len(calls) == 3
    for bad in (dict(x=x[0]), dict(x=x.double()), dict(x=x.t()), dict(x=x[:1].expand(3, 64)), dict(weight=w[:5]), dict(weight=w.double()),
                dict(residual=x[:2]), dict(residual=x.double()), dict(out=x[:, :5]), dict(out=x.bfloat16(), out_dtype=torch.float32),
                dict(group=16), dict(scales=torch.zeros(3, 1)), dict(out_dtype=E4, group=24), dict(out_dtype=E4, group=-16),
                dict(out_dtype=E4, scales=torch.zeros(3, 2)), dict(out_dtype=torch.float64)):
        with pytest.raises(ValueError):
            rms_norm(**{**dict(x=x), **bad})
    assert len(calls) == 3


def test_logprobs_wrapper(calls):
    z, t = torch.zeros(3, 64), torch.zeros(3, dtype=torch.int32)
    assert set(token_logprobs(z, t, top=2)) == {"logprob", "rank", "entropy", "top_ids", "top_logprobs"}
    assert calls == ["moe_token_logprobs"]
    for bad in (dict(logits=z[0]), dict(logits=z.t()), dict(logits=z.double()), dict(tokens=t[:2]), dict(tokens=t.long()), dict(top=-1),
                dict(out={}), dict(out={"entropy": torch.zeros(3), "logprob": torch.zeros(3), "rank": torch.zeros(3)})):
        with pytest.raises(ValueError):
            token_logprobs(**{**dict(logits=z, tokens=t), **bad})


def test_linear_wrapper(calls):
    l = LinearAttention(4, 2, 4, 64, 32, device="cpu")
    q, v, g = torch.zeros(2, 2, 64, dtype=torch.bfloat16), torch.zeros(2, 4, 32, dtype=torch.bfloat16), torch.zeros(2, 4)
    i = lambda *x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    assert l.step(q, q, v, g, slots=i(1, 3)).shape == (2, 4, 32)
    assert l.chunk(q, q, v, g[0], slots=i(1), row_start=i(0, 2)).shape == (2, 4, 32)
    assert calls == ["moe_linear_step", "moe_linear_chunk"]
    ok = dict(q=q, k=q, v=v, g=g, slots=i(0, 1))
    for bad in (dict(q=q.float()), dict(k=q[:, :1]), dict(v=v[:1]), dict(q=q.transpose(1, 2)), dict(g=g.double()), dict(g=g[:1]),
                dict(g=g.t()), dict(slots=i(0, 1).long()), dict(out=v.float()), dict(out=v[:1]), dict(slots=i()),
                dict(v=v[..., ::2])):
        with pytest.raises(ValueError):
            l.step(**{**ok, **bad})
    for bad in (dict(row_start=i(0, 2)), dict(row_start=i()), dict(slots=None, row_start=i(0, 0, 0, 0, 0, 2))):
        with pytest.raises(ValueError):
            l.chunk(**{**ok, **bad})
    for state, Hk, dt in ((torch.zeros(2, 2, 8), 1, torch.bfloat16), (torch.zeros(2, 3, 8, 8), 2, torch.bfloat16),
                          (torch.zeros(2, 2, 8, 8).double(), 1, torch.bfloat16), (torch.zeros(2, 2, 8, 8), 1, torch.float32)):
        with pytest.raises(ValueError):
            LinearAttention.over(state, Hk, dt)
    assert len(calls) == 2


def test_rotary_wrapper(calls, monkeypatch):
    from routed_expert_ffn_router_gb300 import paged
    monkeypatch.setattr(_lib, "moe_workspace_init", lambda *a: None)
    monkeypatch.setattr(paged.PagedKV, "_stream", lambda self, s: 0)
    c = Case([5, 9], [1, 1], 4, 2, 64, 16, dev="cpu")
    kv, r = c.cache(), Rotary(64, device="cpu")
    k = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    assert kv.append_rotary(0, c.q, k, k, r, slots=c.slots).shape == (2, 4, 64) and calls == ["moe_kv_append_rope"]
    p = torch.zeros(2, dtype=torch.int32)
    for bad in (dict(q=c.q[:1]), dict(k=k[:1]), dict(v=k[:, :1]), dict(q=c.q.float()), dict(positions=p[:1]), dict(positions=p.long()),
                dict(q_out=c.q[:1]), dict(q_out=c.q.float()), dict(rotary=Rotary(64, device="meta"))):
        with pytest.raises(ValueError):
            kv.append_rotary(0, **{**dict(q=c.q, k=k, v=k, rotary=r, slots=c.slots), **bad})
    assert len(calls) == 1


def test_calls_refuse_another_device(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1)
    for device in (torch.device("cuda", 0), torch.device("cpu")):
        with pytest.raises(ValueError, match="cuda:1"):
            block._on(device, None)
    assert block._on(torch.device("cuda", 1), 77) == 77


def test_sizes_beyond_int32_are_refused():
    """They would come out modulo 2^32 in the C structs."""
    for shape in ((1 << 31, 1), (1, 1 << 31), (1 << 32, 1)):
        x = torch.zeros(1, dtype=torch.bfloat16).expand(shape)
        with pytest.raises(ValueError, match="more than"):
            rms_norm(x)
        with pytest.raises(ValueError, match="more than"):
            token_logprobs(x)
    layer = LinearAttention(1, 1, 1, 8, 8, device="cpu")
    q = torch.zeros(8, dtype=torch.bfloat16).as_strided((1 << 31, 1, 8), (0, 8, 1))
    with pytest.raises(ValueError, match="fewer than"):
        layer.step(q, q, q, torch.zeros(1))

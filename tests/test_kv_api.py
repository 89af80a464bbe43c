"""The paged cache's C ABI (include/moe_kv.h) refuses bad arguments on the host
before anything is launched, and its Python wrapper checks what it marshals.
No GPU needed."""
import ctypes
import math
import os
import re

import pytest
import torch

from routed_expert_ffn_router_gb300 import _lib
from routed_expert_ffn_router_gb300 import build as libbuild
from routed_expert_ffn_router_gb300.paged import PagedKV
from tests._kv_ref import Books, Case

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INV, UNS, WS, OK = _lib.MOE_ERR_INVALID, _lib.MOE_ERR_UNSUPPORTED, _lib.MOE_ERR_WORKSPACE, _lib.MOE_OK
A = 4096  # an aligned address that nothing touches


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return _lib.load()


def desc(**kw):
    d = _lib.moe_kv_desc()
    base = dict(k=A, v=A, dtype=1, n_layers=2, n_pages=64, page_size=16, Hkv=4, D=128, n_slots=8, max_pages=16,
                table=A, lens=A, refs=A, free_pages=A, n_free=A)
    for n, x in {**base, **kw}.items():
        setattr(d, n, x)
    return d


def rows(**kw):
    r = _lib.moe_kv_rows()
    for n, x in {**dict(B=4, n_rows=4, slots=A, row_start=None), **kw}.items():
        setattr(r, n, x)
    return r


def args(**kw):
    a = _lib.moe_attn_args()
    for n, x in {**dict(Hq=16, scale=0.1, window=0, n_sink=0, q=A, q_stride=16 * 128, o=A, lse=A), **kw}.items():
        setattr(a, n, x)
    return a


def test_every_declared_symbol_is_exported(lib):
    src = open(os.path.join(ROOT, "include", "moe_kv.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    names = set(re.findall(r"\b(moe_[a-z_]+)\s*\(", src))
    assert names == set(_lib.KV_EXPORTS)
    for n in names:
        assert hasattr(lib, n)


BAD_DESC = [
    (dict(k=None), INV), (dict(v=None), INV), (dict(table=None), INV), (dict(lens=None), INV), (dict(refs=None), INV),
    (dict(free_pages=None), INV), (dict(n_free=None), INV), (dict(k=A + 8), INV), (dict(table=A + 2), INV),
    (dict(dtype=0), INV), (dict(dtype=3), INV), (dict(n_layers=0), INV), (dict(n_pages=0), INV),
    (dict(page_size=0), INV), (dict(Hkv=0), INV), (dict(D=0), INV), (dict(n_slots=0), INV), (dict(max_pages=0), INV),
    (dict(D=100), UNS), (dict(D=264), UNS), (dict(max_pages=1 << 21), UNS), (dict(n_slots=1 << 21), UNS),
    (dict(n_pages=1 << 30), UNS), (dict(page_size=1 << 20, max_pages=1 << 12), UNS),
]


@pytest.mark.parametrize("kw,code", BAD_DESC)
def test_bad_descriptions_are_refused_by_every_call(lib, kw, code):
    d = ctypes.byref(desc(**kw))
    big = 1 << 40
    assert lib.moe_kv_workspace_bytes(d, 16, 4) == 0
    assert lib.moe_kv_append(d, 0, ctypes.byref(rows()), A, A, 4 * 128, A, big, None) == code
    for fn in (lib.moe_attn_decode, lib.moe_attn_chunk):
        assert fn(d, 0, ctypes.byref(rows()), ctypes.byref(args()), A, big, None) == code
    assert lib.moe_kv_grow(d, A, A, 1, A, big, None) == code
    assert lib.moe_kv_fork(d, A, A, 1, A, big, None) == code
    assert lib.moe_kv_free(d, A, 1, A, big, None) == code
    assert lib.moe_kv_compact(d, None, A, big, None) == code
    assert lib.moe_kv_copy_pages(d, A, A, 1, A, big, None) == code


@pytest.mark.parametrize("rw,ar,layer,code", [
    (dict(B=-1), {}, 0, INV), (dict(n_rows=-1), {}, 0, INV), (dict(B=0), {}, 0, INV), (dict(n_rows=5), {}, 0, INV),
    (dict(slots=A + 2), {}, 0, INV), ({}, {}, 2, INV), ({}, {}, -1, INV),
    ({}, dict(Hq=0), 0, INV), ({}, dict(Hq=18), 0, INV), ({}, dict(window=-1), 0, INV), ({}, dict(n_sink=-1), 0, INV),
    ({}, dict(scale=math.nan), 0, INV), ({}, dict(scale=math.inf), 0, INV), ({}, dict(q=None), 0, INV),
    ({}, dict(o=None), 0, INV), ({}, dict(q=A + 2), 0, INV), ({}, dict(o=A + 8), 0, INV), ({}, dict(lse=A + 2), 0, INV),
    ({}, dict(q_stride=16 * 128 - 8), 0, INV), ({}, dict(q_stride=16 * 128 + 4), 0, INV),
])
def test_bad_attention_arguments(lib, rw, ar, layer, code):
    for fn in (lib.moe_attn_decode, lib.moe_attn_chunk):
        assert fn(ctypes.byref(desc()), layer, ctypes.byref(rows(**rw)), ctypes.byref(args(**ar)), A, 1 << 40, None) == code


def test_decode_takes_equal_rows_of_at_most_16(lib):
    d, big = ctypes.byref(desc()), 1 << 40
    f = lib.moe_attn_decode
    assert f(d, 0, ctypes.byref(rows(row_start=A)), ctypes.byref(args()), A, big, None) == INV
    assert f(d, 0, ctypes.byref(rows(B=1, n_rows=17)), ctypes.byref(args()), A, big, None) == UNS


def test_workspace(lib):
    d = ctypes.byref(desc())
    need = lib.moe_kv_workspace_bytes(d, 16, 8)
    assert need > 16896 and need % 256 == 0
    assert lib.moe_kv_workspace_bytes(d, 18, 8) == 0 and lib.moe_kv_workspace_bytes(d, 0, 8) == 0
    assert lib.moe_kv_workspace_bytes(d, 16, -1) == 0
    assert lib.moe_kv_workspace_bytes(d, 16, 2048) >= need
    calls = [lambda ws, n: lib.moe_attn_decode(d, 0, ctypes.byref(rows(B=8, n_rows=8)), ctypes.byref(args()), ws, n, None),
             lambda ws, n: lib.moe_attn_chunk(d, 0, ctypes.byref(rows(B=8, n_rows=8)), ctypes.byref(args()), ws, n, None),
             lambda ws, n: lib.moe_kv_grow(d, A, A, 1, ws, n, None), lambda ws, n: lib.moe_kv_fork(d, A, A, 1, ws, n, None),
             lambda ws, n: lib.moe_kv_free(d, A, 1, ws, n, None), lambda ws, n: lib.moe_kv_compact(d, None, ws, n, None),
             lambda ws, n: lib.moe_kv_copy_pages(d, A, A, 1, ws, n, None),
             lambda ws, n: lib.moe_kv_append(d, 0, ctypes.byref(rows()), A, A, 512, ws, n, None)]
    for c in calls:
        assert c(None, need) == WS and c(A + 16, need) == WS and c(A, 16000) == WS


def test_append_and_page_arguments(lib):
    d, big = ctypes.byref(desc()), 1 << 40
    ap = lambda k=A, v=A, st=512, **r: lib.moe_kv_append(d, 0, ctypes.byref(rows(**r)), k, v, st, A, big, None)
    assert ap(k=None) == INV and ap(v=A + 8) == INV and ap(st=504) == INV and ap(st=516) == INV
    assert lib.moe_kv_grow(d, None, A, 1, A, big, None) == INV and lib.moe_kv_grow(d, A, A + 1, 1, A, big, None) == INV
    assert lib.moe_kv_grow(d, A, A, 9, A, big, None) == INV and lib.moe_kv_grow(d, A, A, -1, A, big, None) == INV
    assert lib.moe_kv_fork(d, A, None, 1, A, big, None) == INV and lib.moe_kv_fork(d, A, A, 9, A, big, None) == INV
    assert lib.moe_kv_free(d, None, 1, A, big, None) == INV and lib.moe_kv_free(d, A, 9, A, big, None) == INV
    assert lib.moe_kv_copy_pages(d, A, A, 65, A, big, None) == INV
    assert lib.moe_kv_compact(d, A + 2, A, big, None) == INV


def test_empty_calls_do_nothing(lib):
    d, big = ctypes.byref(desc()), 1 << 40
    none = rows(B=0, n_rows=0, slots=None)
    assert lib.moe_kv_append(d, 0, ctypes.byref(none), None, None, 0, A, big, None) == OK
    for fn in (lib.moe_attn_decode, lib.moe_attn_chunk):
        assert fn(d, 0, ctypes.byref(none), ctypes.byref(args(q=None, o=None)), A, big, None) == OK
    for r in (lib.moe_kv_grow(d, None, None, 0, A, big, None), lib.moe_kv_fork(d, None, None, 0, A, big, None),
              lib.moe_kv_free(d, None, 0, A, big, None), lib.moe_kv_copy_pages(d, None, None, 0, A, big, None)):
        assert r == OK


class _Recorder(PagedKV):
    """A PagedKV over CPU tensors that never reaches the library's GPU calls."""

    def __init__(self, case, max_rows):
        from unittest import mock
        with mock.patch.object(_lib, "moe_workspace_init"):
            self._setup(case.k, case.v, case.table, case.lens, case.refs, case.free, case.n_free, case.Hq, max_rows)


def test_wrapper_checks(lib):
    c = Case([5, 9], [1, 1], 4, 2, 64, 16, dev="cpu")
    kv = _Recorder(c, max_rows=4)
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    for bad in (q.float(), q[:, :3], q.transpose(0, 1).contiguous(), torch.zeros(2, 4, 128, dtype=torch.bfloat16)[:, :, ::2],
                torch.zeros(2, 8, 64, dtype=torch.bfloat16)[:, ::2], torch.zeros(6, 4, 64, dtype=torch.bfloat16)):
        with pytest.raises(ValueError):
            kv.decode(0, bad, slots=c.slots)
    with pytest.raises(ValueError):
        kv.decode(0, q, slots=c.slots.long())
    with pytest.raises(ValueError):
        kv.chunk(0, q, slots=c.slots, row_start=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        kv.decode(0, q, slots=c.slots, out=torch.zeros(2, 4, 64))
    with pytest.raises(ValueError):
        kv.append(0, q[:, :2], torch.zeros(2, 2, 64, dtype=torch.bfloat16), slots=c.slots)  # another row stride
    with pytest.raises(ValueError):
        kv.grow(c.slots, torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        kv.fork(c.slots, torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError):
        PagedKV.over(c.k, c.v.float(), c.table, c.lens, c.refs, c.free, c.n_free)
    with pytest.raises(ValueError):
        PagedKV.over(c.k, c.v, c.table[0], c.lens, c.refs, c.free, c.n_free)


def test_reference_on_worked_values():
    # one key: o = v, lse = scale q.k; equal scores: the mean of v; a window of 1 with one first token
    c = Case([1], [1], 1, 1, 64, 16, dev="cpu")
    o, lse, _, _ = c.reference(scale=0.5)
    pg = int(c.table[int(c.slots[0]), 0])
    assert torch.equal(o[0, 0], c.v[0, pg, 0, 0].double())
    assert abs(float(lse) - 0.5 * float(c.q[0, 0].double() @ c.k[0, pg, 0, 0].double())) < 1e-12
    c = Case([3], [1], 1, 1, 64, 16, window=1, sinks=1, dev="cpu")
    c.q[:] = 0
    pg = int(c.table[int(c.slots[0]), 0])
    o, lse, _, _ = c.reference()
    assert torch.allclose(o[0, 0], (c.v[0, pg, 0, 0].double() + c.v[0, pg, 0, 2].double()) / 2)
    assert abs(float(lse) - math.log(2)) < 1e-12
    # a row before the sequence's first token sees nothing
    o, lse, _, _ = Case([1], [2], 1, 1, 64, 16, dev="cpu").reference()
    assert torch.isneginf(lse[0, 0]) and (o[0] == 0).all() and torch.isfinite(lse[1, 0])


def test_page_books_on_worked_values():
    k = torch.arange(1 * 6 * 1 * 2 * 8).reshape(1, 6, 1, 2, 8).to(torch.bfloat16)
    b = Books(k, k, torch.full((4, 4), -1), torch.zeros(4, dtype=torch.int32), torch.zeros(6, dtype=torch.int32),
              torch.arange(5, -1, -1), 6)
    b.grow([0, 1], [3, 2])                     # slot 0: pages 0, 1; slot 1: page 2
    assert b.table[0][:2] == [0, 1] and b.table[1][0] == 2 and b.stack == [5, 4, 3]
    b.fork([0], [2])                           # page 0 shared, row 0 of page 1 copied to page 3
    assert b.table[2][:2] == [0, 3] and b.refs == [2, 1, 1, 1, 0, 0]
    assert torch.equal(b.k[0, 3, 0, 0], k[0, 1, 0, 0]) and torch.equal(b.k[0, 3, 0, 1], k[0, 3, 0, 1])
    b.free([0])                                # page 1 comes back, page 0 stays
    assert b.refs == [1, 0, 1, 1, 0, 0] and b.stack == [5, 4, 1]
    assert b.compact() == 1                    # page 3 moves to page 1
    assert b.table[2][:2] == [0, 1] and b.stack == [5, 4, 3]

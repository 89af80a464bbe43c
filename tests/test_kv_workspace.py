"""Workspace of the paged cache's calls: what moe_kv_workspace_bytes asks for and
what each call accepts."""
import ctypes

import pytest
import torch

from routed_expert_ffn_router_gb300 import _lib, paged
from routed_expert_ffn_router_gb300 import build as libbuild
from tests._kv_ref import Case, check

A = 4096  # an aligned address that nothing touches


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return _lib.load()


def desc(**kw):
    d = _lib.moe_kv_desc()
    base = dict(k=A, v=A, dtype=1, n_layers=1, n_pages=64, page_size=16, Hkv=1, D=128, n_slots=8, max_pages=8192,
                table=A, lens=A, refs=A, free_pages=A, n_free=A)
    for n, x in {**base, **kw}.items():
        setattr(d, n, x)
    return d


def need(lib, d, Hq, rows):
    return lib.moe_kv_workspace_bytes(ctypes.byref(d), Hq, rows)


def test_decode_partials_are_those_of_one_launch(lib):
    # one launch takes 128 sequences; their partials are all that a call of more needs
    d = desc()
    part = (16 + 8 * 128) * 4  # bytes of a span's sums of 8 query rows
    # tables of 131,072 tokens: at most 256 spans of 64 or 128 tokens, one row of 8
    # heads a sequence, or two in two groups
    assert need(lib, d, 8, 128) == need(lib, d, 8, 128) // 256 * 256
    assert need(lib, d, 8, 2048) <= 16896 + 2 * 128 * 256 * part + 256
    assert need(lib, d, 8, 2048) >= need(lib, d, 8, 128) > need(lib, d, 8, 0)
    small = need(lib, desc(max_pages=4), 8, 0)
    assert need(lib, d, 8, 0) == small  # no rows, no partials: the chunks' region


@pytest.mark.parametrize("kw", [dict(D=80), dict(page_size=24), dict(page_size=4), dict(D=256)])
def test_the_kernel_for_any_size_needs_no_partials(lib, kw):
    d = desc(**kw)
    assert need(lib, d, 8, 2048) == need(lib, d, 8, 0)
    assert need(lib, d, 8, 0) <= 16896 + 4 * (64 + 3 * 64 + 2 * 8) + 256


def test_bytes_grow_with_rows_and_heads(lib):
    for kw in (dict(), dict(Hkv=8, D=64), dict(Hkv=4, page_size=64)):
        d = desc(**kw)
        for Hq in (8, 32):
            sizes = [need(lib, d, Hq, r) for r in (0, 1, 2, 15, 16, 17, 127, 128, 129, 300, 2048)]
            assert sizes == sorted(sizes) and sizes[0] > 0


def test_no_bytes_for_heads_that_no_call_takes(lib):
    a = _lib.moe_attn_args(scale=0.1, q=A, q_stride=1 << 40, o=A)
    for Hkv, Hq in ((1, 65536), (1, 1 << 28), (1, 2 ** 31 - 1), (3, 3 << 29)):
        d, r = desc(Hkv=Hkv), _lib.moe_kv_rows(B=1, n_rows=1, slots=A)
        a.Hq = Hq
        for fn in (lib.moe_attn_decode, lib.moe_attn_chunk):
            assert fn(ctypes.byref(d), 0, ctypes.byref(r), ctypes.byref(a), A, 1 << 60, None) == _lib.MOE_ERR_UNSUPPORTED
        assert need(lib, d, Hq, 16) == 0
    assert need(lib, desc(), 65535, 16) > 0


def test_a_call_with_less_is_refused(lib):
    d = desc(Hkv=2, n_slots=256)
    r = _lib.moe_kv_rows(B=128, n_rows=2048, slots=A)
    a = _lib.moe_attn_args(Hq=16, scale=0.1, q=A, q_stride=16 * 128, o=A)
    ref = ctypes.byref(d), 0, ctypes.byref(r), ctypes.byref(a), A
    assert lib.moe_attn_decode(*ref, need(lib, d, 16, 2048) - 256, None) == _lib.MOE_ERR_WORKSPACE
    assert lib.moe_attn_decode(*ref, need(lib, d, 16, 0), None) == _lib.MOE_ERR_WORKSPACE
    assert lib.moe_attn_chunk(*ref, need(lib, d, 16, 0) - 256, None) == _lib.MOE_ERR_WORKSPACE


def test_max_rows_limits_decode_only(lib, monkeypatch):
    c = Case([9, 9], [6, 6], 4, 2, 64, 16, dev="cpu")
    calls = []
    for name in ("moe_workspace_init", "moe_kv_append", "moe_attn_chunk", "moe_attn_decode"):
        monkeypatch.setattr(_lib, name, lambda *a, name=name: calls.append(name))
    monkeypatch.setattr(paged, "_current_stream", lambda i: 0)
    monkeypatch.setattr(paged, "_current_device", lambda: 0)
    kv = c.cache(max_rows=4)
    calls.clear()
    kv.append(0, c.q[:, :2], c.q[:, :2], slots=c.slots, row_start=c.row_start)
    assert kv.chunk(0, c.q, slots=c.slots, row_start=c.row_start).shape == c.q.shape
    with pytest.raises(ValueError):
        kv.decode(0, c.q, slots=c.slots)
    kv.decode(0, c.q[:4], slots=c.slots)
    assert calls == ["moe_kv_append", "moe_attn_chunk", "moe_attn_decode"]


@pytest.mark.gpu
def test_a_chunk_needs_no_rows_of_decode():
    libbuild.build()
    c = Case([700, 300], [400, 290], 8, 2, 128, 16, torch.bfloat16, 0, 0, seed=61)
    # tables of 131,072 tokens, where decode's partials are the largest part
    c.table = torch.cat([c.table, c.table.new_full((c.n_slots, 8192 - c.max_pages), -1)], 1).contiguous()
    kv = c.cache(max_rows=0)
    bytes0 = need(_lib.load(), kv.desc, 8, 0)
    assert kv.ws_bytes == bytes0 < need(_lib.load(), kv.desc, 8, c.T)
    o, lse = kv.chunk(0, c.q, slots=c.slots, row_start=c.row_start, want_lse=True)
    torch.cuda.synchronize()
    assert kv.status() == (_lib.MOE_OK, 0)
    check(c, (o, lse), c.reference(), "chunk")


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,n", [(8, 1, 1), (8, 1, 2), (4, 2, 4)])
def test_decode_of_more_sequences_than_a_launch_in_the_bytes_asked_for(Hq, Hkv, n):
    lens = [(i * 61) % 400 + 1 for i in range(140)] + [3000, 2100]
    c = Case(lens, [n] * len(lens), Hq, Hkv, 128, 16, torch.bfloat16, 0, 0, seed=62)
    kv = c.cache()
    # what lies after the workspace stays as it is
    guard = torch.full((1 << 20,), 90, dtype=torch.uint8, device="cuda")
    kv.ws = torch.empty(kv.ws_bytes + 256 + guard.numel(), dtype=torch.uint8, device="cuda")
    kv.ws_ptr = kv.ws.data_ptr() + (-kv.ws.data_ptr()) % 256
    end = kv.ws_ptr - kv.ws.data_ptr() + kv.ws_bytes
    kv.ws[end:] = 90
    kv.clear_status()
    o, lse = kv.decode(0, c.q, slots=c.slots, want_lse=True)
    torch.cuda.synchronize()
    assert kv.status() == (_lib.MOE_OK, 0)
    assert bool((kv.ws[end:] == 90).all())
    check(c, (o, lse), c.reference(), "decode")

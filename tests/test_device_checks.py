"""A wrapper refuses a call while another device than its own is current: the
library launches on the current device. No GPU needed (the calls that would
reach one are replaced)."""
import pytest
import torch

from routed_expert_ffn_router_gb300 import _lib, paged
from routed_expert_ffn_router_gb300 import build as libbuild
from routed_expert_ffn_router_gb300.layer import DecodeStack, MoeLayer
from routed_expert_ffn_router_gb300.paged import PagedKV
from tests._kv_ref import Case


@pytest.fixture(scope="module", autouse=True)
def _built():
    libbuild.build()
    _lib.load()


CACHE_CALLS = {
    "moe_kv_append": lambda kv, c: kv.append(0, c.q[:, :2], c.q[:, :2], slots=c.slots),
    "moe_attn_decode": lambda kv, c: kv.decode(0, c.q, slots=c.slots),
    "moe_attn_chunk": lambda kv, c: kv.chunk(0, c.q, slots=c.slots, row_start=c.row_start),
    "moe_kv_grow": lambda kv, c: kv.grow(c.slots, c.slots),
    "moe_kv_fork": lambda kv, c: kv.fork(c.slots, c.slots),
    "moe_kv_free": lambda kv, c: kv.free_slots(c.slots),
    "moe_kv_compact": lambda kv, c: kv.compact(),
    "moe_kv_copy_pages": lambda kv, c: kv.copy_pages(c.slots, c.slots),
    "moe_read_status": lambda kv, c: kv.status(),
    "moe_workspace_init": lambda kv, c: kv.clear_status(),
}


@pytest.mark.parametrize("name", list(CACHE_CALLS))
def test_cache_calls(name, monkeypatch):
    calls = []
    monkeypatch.setattr(_lib, "moe_workspace_init", lambda *a: calls.append("moe_workspace_init"))
    c = Case([5, 9], [1, 1], 4, 2, 64, 16, dev="cpu")
    kv = PagedKV.over(c.k, c.v, c.table, c.lens, c.refs, c.free, c.n_free, Hq=4, max_rows=4)
    calls.clear()
    monkeypatch.setattr(_lib, name, lambda *a: calls.append(name))
    monkeypatch.setattr(paged, "_current_stream", lambda i: 0)
    monkeypatch.setattr(paged, "_current_device", lambda: 1)
    with pytest.raises(ValueError, match="cuda:1"):
        CACHE_CALLS[name](kv, c)
    assert calls == []
    monkeypatch.setattr(paged, "_current_device", lambda: 0)
    CACHE_CALLS[name](kv, c)
    assert calls == [name]


LAYER_CALLS = {
    "moe_layer_forward": lambda o, x: MoeLayer.forward(o, x, x, out=o.out),
    "moe_expert_ffn": lambda o, x: MoeLayer.expert_ffn(o, x, x, x, out=o.out),
    "moe_read_status": lambda o, x: MoeLayer.status(o),
    "moe_workspace_init": lambda o, x: MoeLayer.clear_status(o),
    "moe_decode_stack": lambda o, x: DecodeStack.forward(o),
}


class _Buffers:
    """What the calls above read of a layer or a stack."""
    desc = x_dtype = ws_ptr = ws_bytes = plan_ptr = L = T = outs = None
    T_max = 4
    out = dict.fromkeys(("y", "ids", "w", "miss_ids", "n_miss"))

    class ws:
        device = torch.device("cuda", 0)

    class inp:
        slot_map = None


@pytest.mark.parametrize("name", list(LAYER_CALLS))
def test_layer_calls(name, monkeypatch):
    calls, x = [], torch.zeros(2, 8)
    monkeypatch.setattr(_lib, name, lambda *a: calls.append(name))
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1)
    with pytest.raises(ValueError, match="cuda:1"):
        LAYER_CALLS[name](_Buffers(), x)
    assert calls == []
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    LAYER_CALLS[name](_Buffers(), x)
    assert calls == [name]

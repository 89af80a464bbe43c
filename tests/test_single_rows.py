"""Calls of one row: the distance to a next row, which a slice of a wider tensor keeps,
says nothing and stands in no call's way. No GPU needed."""
import pytest
import torch

from routed_expert_ffn_router_gb300 import _lib, block, linear, paged
from routed_expert_ffn_router_gb300 import build as libbuild
from routed_expert_ffn_router_gb300.block import Rotary, rms_norm, token_logprobs
from routed_expert_ffn_router_gb300.linear import LinearAttention
from tests._kv_ref import Case

BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    libbuild.build()
    _lib.load()


@pytest.fixture
def calls(monkeypatch):
    got = []
    for n in ("moe_rms_norm", "moe_token_logprobs", "moe_linear_step", "moe_linear_chunk", "moe_kv_append_rope", "moe_kv_append",
              "moe_attn_decode", "moe_workspace_init"):
        monkeypatch.setattr(_lib, n, lambda *a: got.append(a))
    for m in (block, linear):
        monkeypatch.setattr(m, "_on", lambda device, stream: 0)
    monkeypatch.setattr(paged.PagedKV, "_stream", lambda self, s: 0)
    return got


def heads(n, D, width):
    """One row of n heads, out of rows of `width` values."""
    return torch.zeros(3, width, dtype=BF)[:, :n * D].unflatten(1, (n, D))[:1]


@pytest.mark.parametrize("op", ["step", "chunk"])
def test_linear(calls, op):
    l = LinearAttention(2, 2, 4, 64, 64, device="cpu")
    q, k, v, g = heads(2, 64, 1001), heads(2, 64, 1003), heads(4, 64, 1005), torch.zeros(1, 7)[:, :4]
    getattr(l, op)(q, k, v, g, slots=torch.tensor([1], dtype=torch.int32))
    a = calls[0][2]._obj
    assert (a.q_stride, a.k_stride, a.v_stride, a.g_stride) == (128, 128, 256, 4)


def test_cache(calls):
    c = Case([5], [1], 4, 2, 64, 16, dev="cpu")
    kv, r = c.cache(), Rotary(64, device="cpu")
    q, k, v = heads(4, 64, 1001), heads(2, 64, 1003), heads(2, 64, 1005)
    calls.clear()
    kv.append_rotary(0, q, k, v, r, slots=c.slots, q_out=heads(4, 64, 777))
    assert (calls[0][7], calls[0][9], calls[0][12]) == (256, 256, 128)
    kv.append(0, k, v, slots=c.slots)
    assert calls[1][5] == 128
    kv.decode(0, q, slots=c.slots)
    assert len(calls) == 3 and kv._args.q_stride == 256


def test_norm_and_logprobs(calls):
    x = torch.zeros(1, 1001, dtype=BF)[:, :64]
    rms_norm(x, residual=torch.zeros(1, 1003, dtype=BF)[:, :64], out=torch.zeros(1, 1005, dtype=BF)[:, :64])
    a = calls[0][0]._obj
    assert (a.x_stride, a.res_stride, a.y_stride) == (64, 64, 64)
    token_logprobs(x)
    assert calls[1][0]._obj.stride == 64


def test_more_rows_keep_their_distance(calls):
    l = LinearAttention(2, 2, 4, 64, 64, device="cpu")
    x = torch.zeros(2, 1008, dtype=BF)
    h = lambda n: x[:, :n * 64].unflatten(1, (n, 64))  # noqa: E731
    l.step(h(2), h(2), h(4), torch.zeros(2, 7)[:, :4])
    a = calls[0][2]._obj
    assert (a.q_stride, a.k_stride, a.v_stride, a.g_stride) == (1008, 1008, 1008, 7)

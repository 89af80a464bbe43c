"""Linear attention with a decay (include/moe_block.h) against the recurrence in
64 bits: decode windows, prompt chunks, and both one after the other."""
import math

import pytest
import torch

from routed_expert_ffn_router_gb300 import build as libbuild
from routed_expert_ffn_router_gb300 import _lib
from routed_expert_ffn_router_gb300.linear import LinearAttention
from tests import _block_ref as ref
from tests._block_ref import within

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16
INF = math.inf


@pytest.fixture(scope="module", autouse=True)
def _built():
    libbuild.build()
    _lib.load()


class Inputs:
    def __init__(self, news, Hk, Hv, Dk, Dv, dtype=BF, seed=0, decay="mixed", n_slots=None, state=True, tail=0):
        g = torch.Generator().manual_seed(seed)
        T = sum(news)
        self.T, self.news, self.dtype = T, list(news), dtype
        self.Hk, self.Hv, self.Dk, self.Dv = Hk, Hv, Dk, Dv
        self.n_slots = len(news) + 2 if n_slots is None else n_slots
        self.slots = torch.randperm(self.n_slots, generator=g)[:len(news)].to(torch.int32).cuda()
        self.start = torch.tensor([0] + list(torch.tensor(news).cumsum(0)), dtype=torch.int32).cuda()

        def part(heads, D, std):  # a part of a wider projection, with rows behind the last sequence
            t = (torch.randn(T + tail, heads * D + 16, generator=g) * std).to(dtype)
            t[T:] = math.nan
            return t.cuda()[:, 8:8 + heads * D].unflatten(1, (heads, D))
        self.q, self.k, self.v = part(Hk, Dk, 1.0), part(Hk, Dk, Dk ** -0.5), part(Hv, Dv, 1.0)
        x = torch.rand(T + tail, Hv, generator=g)
        if decay == "mixed":  # from nearly none to strong, by head
            g0 = -x * torch.logspace(-4, 0.5, Hv)
        elif decay == "none":
            g0 = torch.zeros_like(x)
        elif decay == "strong":
            g0 = -20 * x
        else:  # "resets": some tokens forget all, some decays are above 1 and count as 1
            g0 = torch.where(x < 0.05, torch.full_like(x, -INF), torch.where(x > 0.9, x, -0.1 * x))
        self.g = g0.cuda()
        self.state = (torch.randn(self.n_slots, Hv, Dk, Dv, generator=g) * (1.0 if state else 0.0)).cuda()

    def layer(self):
        return LinearAttention.over(self.state.clone(), self.Hk, self.dtype)

    def spans(self):
        return list(zip(self.slots.tolist(), self.start.tolist(), self.news))

    def want(self, scale, matrix):
        return ref.linear(self.q, self.k, self.v, self.g, self.state, self.spans(), scale, matrix)


def check(i, layer, o, scale, matrix):
    wo, to, ws, ts = i.want(scale, matrix)
    assert layer.status() == 0
    within(o[:i.T], wo[:i.T], to[:i.T], "o")
    within(layer.state, ws, ts, "state")


SHAPES = [  # Hk, Hv, Dk, Dv, dtype
    (16, 32, 128, 128, BF), (4, 4, 64, 64, HF), (2, 6, 64, 128, BF), (1, 2, 128, 64, HF), (1, 3, 256, 256, BF), (2, 2, 8, 8, BF),
    (1, 1, 72, 200, HF), (3, 3, 256, 16, BF), (1, 2, 40, 256, BF),
]


@pytest.mark.parametrize("Hk,Hv,Dk,Dv,dtype", SHAPES)
@pytest.mark.parametrize("B,n", [(1, 1), (3, 1), (5, 2), (2, 16)])
def test_step(Hk, Hv, Dk, Dv, dtype, B, n):
    i = Inputs([n] * B, Hk, Hv, Dk, Dv, dtype, seed=B)
    layer = i.layer()
    check(i, layer, layer.step(i.q, i.k, i.v, i.g, slots=i.slots), Dk ** -0.5, False)


def matrix(i):
    return i.Dk in (64, 128) and i.Dv in (64, 128)


@pytest.mark.parametrize("Hk,Hv,Dk,Dv,dtype", SHAPES)
@pytest.mark.parametrize("news", [[1], [127, 1, 128], [129, 0, 300], [2, 64, 65, 513]])
def test_chunk(Hk, Hv, Dk, Dv, dtype, news):
    i = Inputs(news, Hk, Hv, Dk, Dv, dtype, seed=len(news), tail=3)
    layer = i.layer()
    out = torch.full((i.T + 3, Hv, Dv), 7.0, dtype=dtype, device="cuda")
    layer.chunk(i.q, i.k, i.v, i.g, slots=i.slots, row_start=i.start, out=out)
    assert (out[i.T:] == 7).all()                  # rows behind the last sequence
    check(i, layer, out, Dk ** -0.5, matrix(i))


@pytest.mark.parametrize("decay", ["none", "strong", "resets"])
@pytest.mark.parametrize("D,dtype", [(128, BF), (64, HF), (24, BF)])
def test_decays(decay, D, dtype):
    i = Inputs([150, 260], 2, 4, D, D, dtype, seed=3, decay=decay)
    layer = i.layer()
    o = layer.chunk(i.q, i.k, i.v, i.g, slots=i.slots, row_start=i.start, scale=0.3)
    check(i, layer, o, 0.3, matrix(i))
    j = Inputs([5, 5], 2, 4, D, D, dtype, seed=4, decay=decay)
    layer = j.layer()
    check(j, layer, layer.step(j.q, j.k, j.v, j.g, slots=j.slots, scale=-0.5), -0.5, False)


@pytest.mark.parametrize("D", [128, 64])
def test_long_prompt_few_heads(D):
    """Few heads over a long prompt: the length is what can be split."""
    i = Inputs([3001], 1, 2, D, D, BF, seed=5)
    layer = i.layer()
    check(i, layer, layer.chunk(i.q, i.k, i.v, i.g, slots=i.slots, row_start=i.start), D ** -0.5, True)


@pytest.mark.parametrize("per_head", [True, False])
def test_one_decay_for_all_tokens_and_slots_in_order(per_head):
    i = Inputs([70, 70], 2, 4, 64, 64, BF, seed=6, n_slots=2)
    g = i.g[0].contiguous()
    i.g = g.expand(i.T, -1)
    i.slots = torch.arange(2, dtype=torch.int32).cuda()
    layer = i.layer()
    o = layer.chunk(i.q, i.k, i.v, g if per_head else i.g, row_start=i.start)
    check(i, layer, o, 64 ** -0.5, True)
    j = Inputs([1, 1], 2, 4, 64, 64, BF, seed=7, n_slots=2)
    j.g, j.slots = g.expand(2, -1), i.slots
    layer = j.layer()
    check(j, layer, layer.step(j.q, j.k, j.v, g), 64 ** -0.5, False)


def test_large_values_fp16():
    """Scores and states beyond fp16's range, results within it."""
    i = Inputs([200, 90], 1, 2, 128, 128, HF, seed=8, decay="none", state=False)
    i.q *= 40
    i.k *= 40 * 128 ** 0.5
    i.v += 1
    layer = i.layer()
    s = 2.0 ** -16
    o = layer.chunk(i.q, i.k, i.v, i.g, slots=i.slots, row_start=i.start, scale=s)
    assert float(layer.state.abs().max()) > 1000 and float((i.q[0, 0].double() * i.k[0, 0].double()).sum().abs()) > 10
    check(i, layer, o, s, True)


@pytest.mark.parametrize("op", ["step", "chunk"])
@pytest.mark.parametrize("D", [128, 40])
def test_bad_slots_and_the_same_slot_twice(op, D):
    news = [2, 2, 2, 2]
    i = Inputs(news, 1, 2, D, D, BF, seed=9)
    slots = i.slots.clone()
    slots[1], slots[3] = 99, slots[0]
    layer = i.layer()
    rows = {} if op == "step" else dict(row_start=i.start)
    o = getattr(layer, op)(i.q, i.k, i.v, i.g, slots=slots, **rows)
    assert layer.status() == 2 | 64
    layer.clear_status()
    assert (o[2:4] == 0).all() and (o[6:8] == 0).all()
    wo, to, ws, ts = ref.linear(i.q, i.k, i.v, i.g, i.state, [i.spans()[0], i.spans()[2]], D ** -0.5, op == "chunk" and matrix(i))
    within(o[0:2], wo[0:2], to[0:2], "o")
    within(o[4:6], wo[4:6], to[4:6], "o")
    within(layer.state, ws, ts, "state")
    assert layer.status() == 0


def test_a_prompt_in_pieces_equals_the_whole():
    """Chunks of any cut and single tokens carry the state on."""
    i = Inputs([400], 2, 4, 128, 128, BF, seed=10)
    wo, to, ws, ts = i.want(128 ** -0.5, True)
    for cuts in ([400], [128, 272], [1, 130, 200, 69], [397, 1, 1, 1]):
        layer, at, parts = i.layer(), 0, []
        for n in cuts:
            sl = slice(at, at + n)
            start = torch.tensor([0, n], dtype=torch.int32).cuda()
            if n == 1:
                parts.append(layer.step(i.q[sl], i.k[sl], i.v[sl], i.g[sl], slots=i.slots))
            else:
                parts.append(layer.chunk(i.q[sl], i.k[sl], i.v[sl], i.g[sl], slots=i.slots, row_start=start))
            at += n
        within(torch.cat(parts), wo, to, f"o {cuts}")
        within(layer.state, ws, ts * len(cuts), f"state {cuts}")


def test_no_rows_leave_all_as_it_was():
    i = Inputs([0, 0], 2, 2, 128, 128, BF)
    layer = i.layer()
    e = torch.empty(0, 2, 128, dtype=BF, device="cuda")
    assert layer.chunk(e, e, e, torch.empty(0, 2, device="cuda"), slots=i.slots, row_start=i.start).shape == (0, 2, 128)
    j = Inputs([0, 130, 0], 2, 2, 128, 128, BF, seed=3)
    layer = j.layer()
    o = layer.chunk(j.q, j.k, j.v, j.g, slots=j.slots, row_start=j.start)
    check(j, layer, o, 128 ** -0.5, True)


def test_nan_reaches_its_own_head_only():
    i = Inputs([200, 60], 2, 4, 128, 128, BF, seed=11)
    clean = i.layer()
    want = clean.chunk(i.q, i.k, i.v, i.g, slots=i.slots, row_start=i.start)
    i.v[205, 1] = math.nan
    layer = i.layer()
    o = layer.chunk(i.q, i.k, i.v, i.g, slots=i.slots, row_start=i.start)
    hit = torch.zeros(260, 4, dtype=torch.bool, device="cuda")
    hit[200:, 1] = True
    assert torch.equal(o[~hit], want[~hit]) and torch.isnan(o[205:, 1]).all()
    slot = int(i.slots[1])
    assert torch.isnan(layer.state[slot, 1]).all()
    layer.state[slot, 1] = clean.state[slot, 1]
    assert torch.equal(layer.state, clean.state)


@pytest.mark.parametrize("op", ["step", "chunk"])
def test_streams_graphs_and_repeats(op):
    n = 1 if op == "step" else 300
    i = Inputs([n, n], 4, 8, 128, 128, BF, seed=12)
    rows = {} if op == "step" else dict(row_start=i.start)
    a = i.layer()
    want = getattr(a, op)(i.q, i.k, i.v, i.g, slots=i.slots, **rows)
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        layer = i.layer()
        s.wait_stream(torch.cuda.current_stream())
        got = getattr(layer, op)(i.q, i.k, i.v, i.g, slots=i.slots, stream=stream, **rows)
        s.synchronize()
        assert torch.equal(got, want) and torch.equal(layer.state, a.state)
    layer, graphs = i.layer(), []
    outs = [torch.empty_like(want) for _ in range(2)]
    for o in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            getattr(layer, op)(i.q, i.k, i.v, i.g, slots=i.slots, out=o, **rows)
        graphs.append(g)
    for g, o in zip(graphs, outs):
        layer.state.copy_(i.state)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want) and torch.equal(layer.state, a.state)
    two = [i.layer(), i.layer()]        # two layers' calls at once
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [getattr(l, op)(i.q, i.k, i.v, i.g, slots=i.slots, stream=st, **rows) for l, st in zip(two, streams)]
    torch.cuda.synchronize()
    for l, o in zip(two, got):
        assert torch.equal(o, want) and torch.equal(l.state, a.state)


def test_short_sequences_beside_a_long_one_of_few_heads():
    """The long one is split over a cluster, most of whose CTAs have nothing of the others."""
    i = Inputs([9000, 1, 0, 300, 1200], 1, 1, 64, 64, BF, seed=13)
    layer = i.layer()
    check(i, layer, layer.chunk(i.q, i.k, i.v, i.g, slots=i.slots, row_start=i.start), 64 ** -0.5, True)


def test_many_sequences():
    news = [(7 * j) % 5 for j in range(700)]
    i = Inputs(news, 1, 2, 64, 64, HF, seed=14)
    layer = i.layer()
    check(i, layer, layer.chunk(i.q, i.k, i.v, i.g, slots=i.slots, row_start=i.start), 64 ** -0.5, True)


@pytest.mark.parametrize("value", [math.nan, INF])
def test_padding_may_hold_anything(value):
    """Rows behind the last sequence, and a neighbour's in the same block, reach nothing."""
    i = Inputs([70, 33], 2, 2, 128, 128, BF, seed=15, tail=60)
    for t in (i.q, i.k, i.v):
        t[i.T:] = value
    i.g[i.T:] = value
    layer = i.layer()
    out = torch.zeros(i.T + 60, 2, 128, dtype=BF, device="cuda")
    layer.chunk(i.q, i.k, i.v, i.g, slots=i.slots, row_start=i.start, out=out)
    check(i, layer, out, 128 ** -0.5, True)

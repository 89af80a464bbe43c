"""Calls that the decoder-block operators allow beyond single ones at ordinary sizes:
tensors whose offsets pass 2^31 elements, graphs, several calls at once."""
import pytest
import torch

from routed_expert_ffn_router_gb300 import _lib
from routed_expert_ffn_router_gb300 import build as libbuild
from routed_expert_ffn_router_gb300.block import Rotary, rms_norm, token_logprobs
from routed_expert_ffn_router_gb300.linear import LinearAttention
from tests import _block_ref as ref
from tests._block_ref import within
from tests._kv_ref import Case
from tests.test_linear_gpu import Inputs, check

pytestmark = pytest.mark.gpu
BF, HF, FP, E4 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn
APART, ROWS = (1 << 20) + 16, 2100  # rows so far apart that the last lies beyond 2^31 values


@pytest.fixture(scope="module", autouse=True)
def _built():
    libbuild.build()
    _lib.load()


@pytest.fixture(scope="module")
def far():
    """Two tensors of rows far apart, of which only the first values are ever touched."""
    assert (ROWS - 1) * APART > 1 << 31
    return [torch.empty(ROWS, APART, dtype=BF, device="cuda") for _ in range(2)]


def fill(t, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t.copy_(torch.randn(t.shape, generator=g, device="cuda") * std)
    return t


@pytest.mark.parametrize("out", [BF, E4])
@pytest.mark.parametrize("H", [512, 515])
def test_norm_of_rows_far_apart(far, out, H):
    x, r = fill(far[0][:, :H], 1), fill(far[1][:, :H], 2)
    want_r, y, tol = ref.norm(x, None, r, 1e-6, 0.0, out)
    got = rms_norm(x, residual=r, out_dtype=out)
    assert torch.equal(r, want_r)
    if out is BF:
        within(got, y, tol, "norm")
        rms_norm(r, out=x)
        within(x, *ref.norm(want_r, None, None, 1e-6, 0.0, BF)[1:], "into rows far apart")
        return
    q, s = got[0].double(), got[1].double()
    # half a step of e4m3 relative to the value, of its smallest step below the normal range
    within(q * s, y, tol + (q * s).abs() * 2 ** -4 / (1 - 2 ** -4) + s * 2 ** -10 + y.abs() * 128 * ref.F, "e4m3")


@pytest.mark.parametrize("rows", [ROWS, 40])  # a CTA per row, and clusters of them
def test_logprobs_of_rows_far_apart(far, rows):
    V = 20011
    z = fill(far[0][ROWS - rows:, 3:3 + V], 3, std=3.0)
    tok = (torch.arange(rows, device="cuda") * 7919 % V).int()
    want, tol = ref.logprobs(z, tok, 4, 1.0)
    got = token_logprobs(z, tok, top=4)
    for n in want:
        if n in ("rank", "top_ids"):
            assert torch.equal(got[n], want[n]), n
        else:
            within(got[n], want[n], tol[n], n)


def test_rotary_of_rows_far_apart(far):
    Hq, Hkv, D = 4, 2, 64
    c = Case([ROWS], [ROWS], Hq, Hkv, D, 16, BF, seed=4)
    q = fill(far[0][:, :Hq * D], 4).unflatten(1, (Hq, D))
    k = fill(far[1][:, :Hkv * D], 5).unflatten(1, (Hkv, D))
    v = fill(far[1][:, 4096:4096 + Hkv * D], 6).unflatten(1, (Hkv, D))
    kv, r = c.cache(), Rotary(D)
    pos = torch.arange(ROWS, device="cuda")
    want_q, tol_q = ref.turned(q, pos, r.frequencies, r.gain, D, "half")
    want_k, tol_k = ref.turned(k, pos, r.frequencies, r.gain, D, "half")
    got = kv.append_rotary(0, q, k, v, r, slots=c.slots, row_start=c.row_start, q_out=q)
    u, pg = ref.half_step(BF), c.table[int(c.slots[0])].long()[pos // 16]
    assert kv.status() == (_lib.MOE_OK, 0)
    within(got, want_q, tol_q + u * want_q.abs(), "q")
    within(c.k[0, pg, :, pos % 16], want_k, tol_k + u * want_k.abs(), "k")
    assert torch.equal(c.v[0, pg, :, pos % 16], v)


@pytest.mark.parametrize("op", ["step", "chunk"])
@pytest.mark.parametrize("D", [128, 72])
def test_linear_of_rows_and_states_far_apart(far, op, D):
    """Rows of a projection far apart, and the last slots of 2^31 values of state and more."""
    n_slots = (1 << 31) // (4 * D * D) + 40
    state = torch.empty(n_slots, 4, D, D, device="cuda")
    assert state.numel() > 1 << 31
    news = [1] * ROWS if op == "step" else [ROWS - 300, 300]
    if op == "step":
        news = [1] * 30
    i = Inputs(news, 2, 4, D, D, BF, seed=6, n_slots=len(news))
    at = ROWS - i.T
    rows = lambda t, b, o: far[b][at:, o:o + t[0].numel()].unflatten(1, t.shape[1:]).copy_(t)  # noqa: E731
    i.q, i.k, i.v = rows(i.q, 0, 0), rows(i.k, 1, 0), rows(i.v, 1, 8192)
    last = torch.arange(n_slots - len(news), n_slots, device="cuda")
    state[last] = i.state
    layer = LinearAttention.over(state, 2)
    call = dict(slots=(i.slots + (n_slots - len(news))).int())
    if op == "chunk":
        call["row_start"] = i.start
    o = getattr(layer, op)(i.q, i.k, i.v, i.g, **call)
    assert layer.status() == 0
    wo, to, ws, ts = i.want(D ** -0.5, op == "chunk" and D == 128)
    within(o, wo, to, "o")
    within(state[last], ws, ts, "state")


def test_rotary_append_in_graphs_and_on_other_streams():
    c = Case([40, 1, 133], [17, 1, 60], 8, 2, 128, 16, BF, seed=7)
    kv, r = c.cache(), Rotary(128)
    g = torch.Generator(device="cuda").manual_seed(8)
    k, v = (torch.randn(c.T, 2, 128, generator=g, device="cuda").to(BF) for _ in range(2))
    pools = lambda: (c.k.view(torch.int16).clone(), c.v.view(torch.int16).clone())  # noqa: E731
    before = c.k.clone(), c.v.clone()

    def again():
        c.k.copy_(before[0])
        c.v.copy_(before[1])
    rows = dict(slots=c.slots, row_start=c.row_start)
    want = kv.append_rotary(0, c.q, k, v, r, **rows)
    after = pools()
    same = lambda: all(torch.equal(a, b) for a, b in zip(pools(), after))  # noqa: E731
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        again()
        s.wait_stream(torch.cuda.current_stream())
        got = kv.append_rotary(0, c.q, k, v, r, stream=stream, **rows)
        s.synchronize()
        assert torch.equal(got, want) and same()
    graph, out = torch.cuda.CUDAGraph(), torch.empty_like(want)
    with torch.cuda.graph(graph):
        kv.append_rotary(0, c.q, k, v, r, q_out=out, **rows)
    for _ in range(2):
        again()
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and same()
    # another length, as a replayed step finds it: the graph goes by what the tensors hold
    c.lens[int(c.slots[1])] = 5
    c.table[int(c.slots[1]), 0] = int(c.free[0])
    again()
    graph.replay()
    torch.cuda.synchronize()
    w, tol = ref.turned(c.q[17:18], torch.tensor([4], device="cuda"), r.frequencies, r.gain, 128, "half")
    within(out[17:18], w, tol + ref.half_step(BF) * w.abs(), "q of the longer sequence")
    assert torch.equal(out[:17], want[:17]) and torch.equal(out[18:], want[18:])
    assert torch.equal(c.v[0, int(c.free[0]), :, 4], v[17])


def test_divided_prompts_in_graphs_and_at_once():
    """Sequences divided over clusters: two layers' calls on two streams, and two graphs."""
    i = Inputs([1500], 2, 4, 128, 128, BF, seed=9)
    rows = dict(slots=i.slots, row_start=i.start)
    first = i.layer()
    want = first.chunk(i.q, i.k, i.v, i.g, **rows)
    check(i, first, want, 128 ** -0.5, True)
    layers, streams = [i.layer() for _ in range(4)], [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    got = [l.chunk(i.q, i.k, i.v, i.g, stream=s, **rows) for l, s in zip(layers, streams)]
    torch.cuda.synchronize()
    for l, o in zip(layers, got):
        assert torch.equal(o, want) and torch.equal(l.state, first.state) and l.status() == 0
    graphs, outs = [], [torch.empty_like(want) for _ in range(2)]
    for l, o in zip(layers, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            l.chunk(i.q, i.k, i.v, i.g, out=o, **rows)
        graphs.append(g)
    for _ in range(3):
        for l in layers[:2]:
            l.state.copy_(i.state)
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for l, o in zip(layers, outs):
            assert torch.equal(o, want) and torch.equal(l.state, first.state)


def test_logprobs_and_norms_at_once():
    g = torch.Generator(device="cuda").manual_seed(10)
    z = torch.randn(40, 50257, generator=g, device="cuda").to(BF)
    tok = torch.arange(40, dtype=torch.int32, device="cuda")
    x = torch.randn(3000, 1024, generator=g, device="cuda").to(BF)
    want, y = token_logprobs(z, tok, top=9), rms_norm(x)
    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [(token_logprobs(z, tok, top=9, stream=s), rms_norm(x, stream=s)) for s in streams]
        torch.cuda.synchronize()
        for r, h in got:
            assert all(torch.equal(r[n], want[n]) for n in want) and torch.equal(h, y)

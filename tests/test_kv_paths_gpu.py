"""Paths of the paged cache's attention that need many sequences, many items, a
wide table or few rows over a long one to be taken, against the 64-bit
definition."""
import pytest
import torch

from routed_expert_ffn_router_gb300 import _lib
from routed_expert_ffn_router_gb300 import build as libbuild
from tests._kv_ref import Case, check

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _built():
    libbuild.build()
    _lib.load()


def run(c, op, kv=None, **kw):
    kv = c.cache() if kv is None else kv
    ms = dict(window=c.window, sinks=c.sinks, want_lse=True)
    if op == "decode":
        out = kv.decode(0, c.q, slots=c.slots, **ms, **kw)
    else:
        out = kv.chunk(0, c.q, slots=c.slots, row_start=c.row_start, **ms, **kw)
    torch.cuda.synchronize()
    assert kv.status() == (_lib.MOE_OK, 0)
    return out


def widen(c, tokens):
    """A table for sequences of up to `tokens` tokens, garbage past the lengths."""
    more = tokens // c.page - c.max_pages
    c.table = torch.cat([c.table, torch.full((c.n_slots, more), 1 << 30, dtype=torch.int32, device=c.dev)], 1).contiguous()
    c.max_pages += more


@pytest.mark.parametrize("n,D", [(1, 128), (4, 64)])
def test_decode_items_beyond_the_ctas_split_and_joined(n, D):
    # 8 KV heads of 64 sequences are more items than any grid; the long ones lie in
    # many CTAs each. A row's bits are those of its sequence alone.
    lens = [(i * 131) % 700 + 1 for i in range(60)] + [30011, 9000, 5003, 17000]
    c = Case(lens, [n] * 64, 16, 8, D, 32, BF, 0, 0, seed=71)
    kv = c.cache()
    o, lse = run(c, "decode", kv)
    check(c, (o, lse), c.reference(), "decode")
    for b in (0, 7, 59, 60, 61, 63):
        ob, lb = kv.decode(0, c.q[n * b:n * b + n], slots=c.slots[b:b + 1], want_lse=True)
        assert torch.equal(ob, o[n * b:n * b + n]) and torch.equal(lb, lse[n * b:n * b + n]), b


@pytest.mark.parametrize("B", [128, 129, 300])
@pytest.mark.parametrize("n,window,sinks", [(1, 0, 0), (3, 50, 2)])
def test_decode_in_several_launches(B, n, window, sinks):
    lens = [(i * 37) % 260 for i in range(B)]
    c = Case(lens, [n] * B, 4, 2, 128, 16, BF, window, sinks, seed=72)
    o, lse = run(c, "decode")
    check(c, (o, lse), c.reference(), "decode")
    # without slots, sequence b is slot b
    q = torch.zeros(c.n_slots, n, 4, 128, dtype=BF, device="cuda")
    q[c.slots.long()] = c.q.reshape(B, n, 4, 128)
    idle = torch.ones(c.n_slots, dtype=torch.bool, device="cuda")
    idle[c.slots.long()] = False
    kv = c.cache(max_rows=c.n_slots * n)
    slots = torch.arange(c.n_slots, dtype=torch.int32, device="cuda")
    want = kv.decode(0, q.flatten(0, 1), slots=slots, window=window, sinks=sinks, want_lse=True)
    torch.cuda.synchronize()
    assert kv.status() == (_lib.MOE_OK, 0)
    at = (c.slots.long()[:, None] * n + torch.arange(n, device="cuda")).flatten()
    assert torch.equal(want[0][at], o) and torch.equal(want[1][at], lse)
    if n == 1:  # the wrapper takes a row per slot without slots
        got = kv.decode(0, q.flatten(0, 1), window=window, sinks=sinks, want_lse=True)
        torch.cuda.synchronize()
        assert kv.status() == (_lib.MOE_OK, 0)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert (got[0][idle] == 0).all() and torch.isneginf(got[1][idle]).all()


@pytest.mark.parametrize("op", ["decode", "chunk"])
def test_a_slot_out_of_range_in_a_later_launch(op):
    B = 300
    c = Case([(i * 37) % 90 + 1 for i in range(B)], [1] * B, 4, 2, 64, 16, BF, 0, 0, seed=73)
    kv = c.cache()
    o, lse = run(c, op, kv)
    slots = c.slots.clone()
    slots[290] = c.n_slots
    got = kv.decode(0, c.q, slots=slots, want_lse=True) if op == "decode" else \
        kv.chunk(0, c.q, slots=slots, row_start=c.row_start, want_lse=True)
    torch.cuda.synchronize()
    assert kv.status() == (_lib.MOE_ERR_DEVICE, 2)
    rest = torch.arange(B, device="cuda") != 290
    assert (got[0][290] == 0).all() and torch.isneginf(got[1][290]).all()
    if op == "decode":
        assert torch.equal(got[0][rest], o[rest]) and torch.equal(got[1][rest], lse[rest])
    else:
        ro, rl, to, tl = c.reference()
        assert ((got[0].double() - ro).abs() <= to)[rest].all() and ((got[1].double() - rl).abs() <= tl)[rest].all()


@pytest.mark.parametrize("B", [256, 257, 600])
@pytest.mark.parametrize("D", [64, 128])
def test_chunks_in_several_launches(B, D):
    lens = [(i * 37) % 200 for i in range(B)]
    news = [min(n, (i * 11) % 7) for i, n in enumerate(lens)]
    c = Case(lens, news, 4, 2, D, 16, BF, 0, 0, seed=74)
    check(c, run(c, "chunk"), c.reference(), "chunk")


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("lens,news,Hq,Hkv,window,sinks", [
    ([6000], [20], 8, 2, 0, 0), ([6000, 3000], [33, 2], 8, 2, 2500, 4), ([4000, 2300, 9], [1, 130, 9], 28, 4, 0, 0),
])
@pytest.mark.parametrize("D", [64, 128])
def test_few_rows_over_a_long_context(D, lens, news, Hq, Hkv, window, sinks, dtype):
    # units in many CTAs, whose parts the kernel after it joins
    c = Case(lens, news, Hq, Hkv, D, 64, dtype, window, sinks, seed=75)
    kv = c.cache()
    o, lse = run(c, "chunk", kv)
    check(c, (o, lse), c.reference(), "chunk")
    again = run(c, "chunk", kv)
    assert torch.equal(again[0], o) and torch.equal(again[1], lse)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens,news", [([40], [40]), ([1], [1]), ([300, 5, 0, 129], [300, 5, 0, 2]), ([700], [640])])
@pytest.mark.parametrize("op", ["decode", "chunk"])
def test_a_wide_table_over_short_sequences(op, lens, news, D):
    news = [2] * len(lens) if op == "decode" else news
    c = Case(lens, news, 16, 4, D, 16, FP, 0, 0, seed=76)
    tight = run(c, op)
    widen(c, 32768)
    wide = run(c, op)
    check(c, wide, c.reference(), op)
    if op == "decode":
        assert torch.equal(wide[0], tight[0]) and torch.equal(wide[1], tight[1])


def test_chunk_rows_next_to_other_sequences_and_alone():
    lens, news = [900, 300, 64, 2500], [300, 300, 17, 60]
    c = Case(lens, news, 8, 2, 128, 16, BF, 200, 4, seed=77)
    kv = c.cache()
    check(c, run(c, "chunk", kv), c.reference(), "together")
    ro, rl, to, tl = c.reference()
    start = c.row_start.tolist()
    for b in range(4):
        rows = slice(start[b], start[b + 1])
        o, lse = kv.chunk(0, c.q[rows], slots=c.slots[b:b + 1], row_start=c.row_start.new_tensor([0, news[b]]), window=200,
                          sinks=4, want_lse=True)
        assert ((o.double() - ro[rows]).abs() <= to[rows]).all() and ((lse.double() - rl[rows]).abs() <= tl[rows]).all(), b


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("Hq,Hkv,n,D,page", [(4, 2, 1, 128, 16), (8, 1, 2, 64, 16), (4, 2, 1, 80, 16)])
def test_decode_probabilities_are_not_rounded_to_the_type(Hq, Hkv, n, D, page, dtype):
    """Half the keys have probability 1 and the value -w, the others the probability r,
    which the type does not hold, and the value 1, with w = r rounded: the result is what
    that rounding would lose. Against a bound with the squared half step, of a probability
    as two values of the type."""
    u = torch.finfo(dtype).eps / 2
    s = -0.58984375 if dtype == FP else -0.62890625
    r = float(torch.tensor(s, dtype=torch.float64).exp())
    w = float(torch.tensor(r).to(dtype))
    assert abs(r - w) / r > u / 4
    c = Case([128], [n], Hq, Hkv, D, page, dtype, 0, 0, seed=78, poison=False)
    c.q.zero_()
    c.k.zero_()
    c.q[..., 0] = 1.0
    c.k[..., 0::2, 0] = s
    c.v[..., 0::2, :] = 1.0
    c.v[..., 1::2, :] = -w
    ro, rl, to, tl = c.reference(scale=1.0)
    v = c.v
    c.v = v.abs()
    A = c.reference(scale=1.0)[0]
    c.v = v
    to = to - 1.05 * (u - u * u) * A
    assert (to[-1] < ro[-1].abs() / 2).all()  # (the bound is below what a rounding would lose)
    check(c, run(c, "decode", scale=1.0), (ro, rl, to, tl), "decode")

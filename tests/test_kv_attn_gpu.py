"""Attention over the paged cache on the GPU against the 64-bit definition:
decode windows and prompt chunks, at the sizes, masks and layouts where they
can go wrong. Everything no row may use is NaN or a garbage page number."""
import math

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


# lens, rows per sequence, Hq, Hkv, D, page, dtype, window, sinks
DECODE = {
    "one_token": ([1], 1, 4, 2, 128, 16, BF, 0, 0),
    "empty_and_short": ([0, 1, 2, 15, 16, 17, 0], 1, 8, 2, 128, 16, BF, 0, 0),
    "tile_edges": ([63, 64, 65, 127, 128, 129, 255, 256, 257], 1, 16, 4, 64, 32, FP, 0, 0),
    "rows_before_the_first_token": ([0, 1, 2, 3, 40], 3, 4, 4, 128, 16, BF, 0, 0),
    "mqa_24_heads": ([100, 33], 1, 24, 1, 128, 16, BF, 0, 0),
    "pairs_of_8": ([300, 65, 64, 2], 2, 32, 4, 128, 16, FP, 0, 0),
    "sixteen_rows": ([70, 16, 3], 16, 8, 2, 64, 64, BF, 0, 0),
    "mha_odd_heads": ([200, 31], 1, 5, 5, 64, 16, BF, 0, 0),
    "groups_of_7": ([511, 90], 2, 28, 4, 128, 32, BF, 0, 0),
    "window": ([1000, 64, 10, 129], 1, 8, 2, 128, 16, BF, 64, 0),
    "window_one": ([77, 1, 64, 65], 1, 8, 2, 128, 16, FP, 1, 0),
    "window_sinks": ([1000, 700, 37, 130, 128], 2, 8, 2, 128, 32, BF, 100, 4),
    "sinks_meet_window": ([200, 101, 100, 99], 1, 8, 2, 64, 16, BF, 64, 37),
    "sinks_longer_than_window": ([900, 100], 3, 8, 2, 128, 16, BF, 5, 130),
    "many_rows_window": ([400, 20], 16, 16, 2, 128, 16, BF, 7, 3),
    "long": ([9001, 4097, 4096], 1, 8, 2, 128, 64, BF, 0, 0),
    "long_pairs": ([20011], 2, 16, 2, 64, 16, FP, 0, 0),
    "page_8": ([100, 8, 9], 1, 8, 2, 128, 8, BF, 0, 0),
    "page_128": ([300, 128, 129], 1, 8, 2, 128, 128, BF, 0, 0),
    "page_256": ([700, 1], 2, 8, 2, 64, 256, FP, 0, 0),
    "page_1": ([37, 2], 1, 4, 2, 128, 1, BF, 0, 0),
    "page_24": ([100, 24, 25], 1, 4, 2, 64, 24, BF, 30, 2),
    "d80": ([100, 3], 2, 4, 2, 80, 16, FP, 0, 0),
    "d256": ([300, 64], 1, 8, 2, 256, 16, BF, 90, 4),
    "d8": ([50], 1, 2, 1, 8, 16, BF, 0, 0),
    "batch": ([(i * 97) % 530 + 1 for i in range(60)], 1, 16, 2, 128, 16, BF, 0, 0),
}


@pytest.mark.parametrize("name", list(DECODE))
def test_decode(name):
    lens, n, Hq, Hkv, D, page, dt, W, S = DECODE[name]
    c = Case(lens, [n] * len(lens), Hq, Hkv, D, page, dt, W, S, seed=len(name))
    check(c, run(c, "decode"), c.reference(), name)


# lens, news, Hq, Hkv, D, page, dtype, window, sinks
CHUNK = {
    "one": ([1], [1], 4, 2, 128, 16, BF, 0, 0),
    "short": ([40], [40], 16, 4, 64, 16, FP, 0, 0),
    "empty_sequences": ([0, 5, 0, 130], [0, 5, 0, 130], 8, 2, 128, 16, BF, 0, 0),
    "no_new_rows": ([50, 20], [0, 20], 8, 2, 128, 16, BF, 0, 0),
    "rows_before_the_first_token": ([3, 0], [7, 4], 8, 2, 64, 16, BF, 0, 0),
    "tile_edges": ([127, 128, 129, 255], [127, 128, 129, 255], 4, 4, 128, 16, BF, 0, 0),
    "context": ([700], [130], 8, 2, 128, 32, BF, 0, 0),
    "context_ragged": ([513, 300, 129, 64], [1, 200, 129, 3], 16, 4, 128, 16, FP, 0, 0),
    "mqa_24": ([150], [150], 24, 1, 128, 16, BF, 0, 0),
    "groups_of_7": ([333, 100], [70, 100], 28, 4, 64, 32, BF, 0, 0),
    "groups_of_3": ([300], [299], 12, 4, 128, 16, BF, 0, 0),
    "mha": ([260, 40], [260, 39], 5, 5, 64, 16, BF, 0, 0),
    "window": ([600], [600], 8, 2, 128, 16, BF, 100, 0),
    "window_one": ([150], [150], 4, 2, 64, 16, FP, 1, 0),
    "window_sinks": ([900, 333], [400, 333], 8, 2, 128, 32, BF, 200, 4),
    "window_far_from_sinks": ([1500], [140], 8, 2, 128, 16, BF, 64, 37),
    "window_exact_tile": ([1024], [256], 8, 4, 128, 16, BF, 128, 128),
    "sinks_longer_than_window": ([700], [300], 8, 2, 64, 64, BF, 10, 300),
    "page_8": ([200], [150], 4, 2, 128, 8, BF, 0, 0),
    "page_128": ([400], [200], 8, 2, 128, 128, BF, 0, 0),
    "page_256": ([400], [200], 8, 2, 64, 256, FP, 90, 3),
    "page_24": ([100], [90], 4, 2, 64, 24, BF, 0, 0),
    "d80": ([100], [100], 4, 2, 80, 16, FP, 0, 0),
    "d256": ([200], [150], 4, 2, 256, 16, BF, 0, 0),
    "long_context_few_rows": ([6000], [20], 8, 2, 128, 64, BF, 0, 0),
    "long_context_few_rows_window": ([6000, 3000], [33, 2], 8, 2, 128, 64, FP, 2500, 4),
    "big": ([1100], [1024], 16, 4, 128, 16, BF, 0, 0),
    "many": ([(i * 53) % 300 + 20 for i in range(20)], [(i * 29) % 20 + 1 for i in range(20)], 8, 2, 128, 16, BF, 0, 0),
}


@pytest.mark.parametrize("name", list(CHUNK))
def test_chunk(name):
    lens, news, Hq, Hkv, D, page, dt, W, S = CHUNK[name]
    c = Case(lens, news, Hq, Hkv, D, page, dt, W, S, seed=len(name))
    check(c, run(c, "chunk"), c.reference(), name)


@pytest.mark.parametrize("op", ["decode", "chunk"])
@pytest.mark.parametrize("gain,mean", [(0.0, 0.0), (40.0, 0.0), (1.5, 30.0)])
def test_flat_peaked_and_offset_values(op, gain, mean):
    # equal scores; one key takes everything; values far from zero
    n = 2 if op == "decode" else 150
    c = Case([300, 170], [n, n], 8, 2, 128, 16, BF, 0, 0, seed=5, q_gain=gain, v_mean=mean)
    check(c, run(c, op), c.reference(), op)


@pytest.mark.parametrize("op", ["decode", "chunk"])
@pytest.mark.parametrize("scale", [0.0, -0.2, 1.0])
def test_scale(op, scale):
    n = 1 if op == "decode" else 60
    c = Case([200], [n], 8, 2, 64, 16, FP, 0, 0, seed=7)
    check(c, run(c, op, scale=scale), c.reference(scale=scale), op)


@pytest.mark.parametrize("D", [64, 128])
def test_decode_value_that_is_not_finite_stays_with_the_rows_that_see_it(D):
    # the newest token's value is infinite or NaN: the row before it does not see it
    for bad in (math.inf, math.nan):
        c = Case([70, 64, 65], [2, 2, 2], 8, 2, D, 16, BF, 0, 0, seed=3)
        for b, s in enumerate(c.slots.tolist()):
            L = c.lens_l[b]
            c.v[0, int(c.table[s, (L - 1) // 16]), :, (L - 1) % 16, 5] = bad
        o, lse = run(c, "decode")
        ro, rl, to, tl = c.reference()
        assert torch.isfinite(o[0::2]).all()
        assert not torch.isfinite(o[1::2, :, 5]).any()
        check(c, (o, lse), (ro, rl, to, tl), "not finite")


def test_decode_row_does_not_depend_on_the_other_sequences():
    lens = [5000, 3, 700, 64, 129, 2049, 1, 33]
    c = Case(lens, [2] * 8, 16, 2, 128, 16, BF, 0, 0, seed=11)
    kv = c.cache()
    o, lse = run(c, "decode", kv)
    for b in range(8):
        ob, lb = kv.decode(0, c.q[2 * b:2 * b + 2], slots=c.slots[b:b + 1], want_lse=True)
        assert torch.equal(ob, o[2 * b:2 * b + 2]) and torch.equal(lb, lse[2 * b:2 * b + 2]), b
    again = run(c, "decode", kv)
    assert torch.equal(again[0], o) and torch.equal(again[1], lse)


def test_chunk_is_deterministic_and_rows_do_not_depend_on_other_sequences():
    lens, news = [900, 300, 64], [300, 300, 17]
    c = Case(lens, news, 8, 2, 128, 16, BF, 200, 4, seed=12)
    kv = c.cache()
    o, lse = run(c, "chunk", kv)
    again = run(c, "chunk", kv)
    assert torch.equal(again[0], o) and torch.equal(again[1], lse)


@pytest.mark.parametrize("op", ["decode", "chunk"])
def test_on_another_stream_and_in_a_graph(op):
    n = 1 if op == "decode" else 100
    c = Case([300, 200], [n, n], 8, 2, 128, 16, BF, 0, 0, seed=13)
    kv = c.cache()
    want = run(c, op, kv)
    s = torch.cuda.Stream()
    o, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    s.wait_stream(torch.cuda.current_stream())
    call = (lambda: kv.decode(0, c.q, slots=c.slots, out=o, lse=lse)) if op == "decode" else \
        (lambda: kv.chunk(0, c.q, slots=c.slots, row_start=c.row_start, out=o, lse=lse))
    with torch.cuda.stream(s):
        call()
    s.synchronize()
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    # a replay reads the lengths of the moment: one token fewer
    c.lens -= (c.lens > 0).int()
    o.fill_(7)
    g.replay()
    torch.cuda.synchronize()
    ref = kv.decode(0, c.q, slots=c.slots, want_lse=True) if op == "decode" else \
        kv.chunk(0, c.q, slots=c.slots, row_start=c.row_start, want_lse=True)
    torch.cuda.synchronize()
    assert torch.equal(o, ref[0]) and torch.equal(lse, ref[1])
    assert not torch.equal(o, want[0])


@pytest.mark.parametrize("op", ["decode", "chunk"])
def test_bad_pages_and_slots_are_reported(op):
    n = 1 if op == "decode" else 40
    c = Case([100, 90], [n, n], 8, 2, 128, 16, BF, 0, 0, seed=14)
    kv = c.cache()
    s0, s1 = c.slots.tolist()
    c.table[s0, 2] = c.n_pages          # tokens 32 .. 47 of the first sequence
    call = lambda sl: kv.decode(0, c.q, slots=sl, want_lse=True) if op == "decode" else \
        kv.chunk(0, c.q, slots=sl, row_start=c.row_start, want_lse=True)
    o, lse = call(c.slots)
    torch.cuda.synchronize()
    code, bits = kv.status()
    assert code == _lib.MOE_ERR_DEVICE and bits == 2
    assert torch.isfinite(o).all()      # the bad page's tokens are left out
    kv.clear_status()
    sl = torch.tensor([c.n_slots, s1], dtype=torch.int32, device="cuda")
    o2, lse2 = call(sl)
    torch.cuda.synchronize()
    assert kv.status() == (_lib.MOE_ERR_DEVICE, 2)
    assert (o2[:n] == 0).all() and torch.isneginf(lse2[:n]).all()
    assert torch.equal(o2[n:], o[n:]) and torch.equal(lse2[n:], lse[n:])
    kv.clear_status()
    # a length beyond the table's width is taken as the width
    c.lens[s1] = 10 ** 9
    call(sl[1:].repeat(2).contiguous())
    torch.cuda.synchronize()
    assert kv.status()[1] == 2


def test_without_slots_and_without_lse():
    c = Case([90, 40, 70], [1, 1, 1], 8, 2, 128, 16, BF, 0, 0, seed=15)
    kv = c.cache(max_rows=c.n_slots)
    want = run(c, "decode", kv)[0]
    # without slots, sequence b is slot b: a row for every slot, some of them empty
    q = torch.zeros(c.n_slots, 8, 128, dtype=BF, device="cuda")
    q[c.slots.long()] = c.q
    got = kv.decode(0, q)
    torch.cuda.synchronize()
    assert kv.status() == (_lib.MOE_OK, 0)
    assert torch.equal(got[c.slots.long()], want)
    idle = torch.ones(c.n_slots, dtype=torch.bool, device="cuda")
    idle[c.slots.long()] = False
    assert (got[idle] == 0).all()


def test_pools_beyond_2_to_the_32_elements():
    page, Hkv, D = 64, 8, 128
    n_pages = (1 << 32) // (page * Hkv * D) + 40
    from routed_expert_ffn_router_gb300.paged import PagedKV
    k = torch.empty(1, n_pages, Hkv, page, D, dtype=BF, device="cuda")
    v = torch.empty_like(k)
    c = Case([200, 130], [1, 1], 16, Hkv, D, page, BF, 0, 0, seed=16, spare_pages=0)
    last = n_pages - c.n_pages
    k[:, last:], v[:, last:] = c.k, c.v
    c.k, c.v = k, v
    c.table = torch.where((c.table >= 0) & (c.table < c.n_pages), c.table + last, c.table)
    refs = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    kv = PagedKV.over(k, v, c.table, c.lens, refs, torch.zeros_like(refs), c.n_free, Hq=16, max_rows=300)
    check(c, run(c, "decode", kv), c.reference(), "decode")
    c2 = Case([200, 130], [120, 77], 16, Hkv, D, page, BF, 0, 0, seed=16, spare_pages=0)
    k[:, last:], v[:, last:] = c2.k, c2.v
    c2.table = torch.where((c2.table >= 0) & (c2.table < c2.n_pages), c2.table + last, c2.table)
    c2.k, c2.v = k, v
    kv = PagedKV.over(k, v, c2.table, c2.lens, refs, torch.zeros_like(refs), c2.n_free, Hq=16, max_rows=300)
    check(c2, run(c2, "chunk", kv), c2.reference(), "chunk")
    del k, v
    torch.cuda.empty_cache()


# lens, rows, page, window, sinks: boxes of first tokens and of the window packed into one block
PACKED = {
    "page_8": ([700, 333], [150, 40], 8, 130, 5),
    "page_64": ([900, 400], [200, 90], 64, 200, 70),
    "page_128": ([900, 257], [130, 257], 128, 100, 3),
    "page_256": ([1200, 513], [300, 100], 256, 260, 300),
    "first_tokens_end_a_box": ([640, 640], [70, 1], 32, 96, 64),
    "first_tokens_meet_window": ([300, 300], [64, 33], 16, 200, 90),
    "one_key_windows": ([500], [129], 16, 1, 129),
    "window_longer_than_the_sequence": ([200, 90], [200, 17], 32, 512, 4),
}


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("name", list(PACKED))
def test_chunk_blocks_of_first_tokens_and_window(name, D):
    lens, news, page, window, sinks = PACKED[name]
    c = Case(lens, news, 14, 2, D, page, BF, window, sinks, seed=31)
    check(c, run(c, "chunk"), c.reference(), name)


@pytest.mark.parametrize("op,lens,news,Hq,Hkv,D,page,window,sinks", [
    ("decode", [2100, 1, 0, 65], [3, 3, 3, 3], 6, 2, 80, 16, 0, 0),
    ("decode", [1500, 70], [1, 1], 4, 4, 72, 24, 700, 11),
    ("decode", [900, 4097], [2, 2], 8, 2, 128, 20, 0, 0),
    ("decode", [333], [16], 4, 1, 256, 7, 50, 60),
    ("chunk", [1000, 3], [40, 3], 6, 2, 80, 16, 300, 4),
    ("chunk", [700], [700], 12, 3, 40, 12, 0, 0),
])
def test_any_head_and_page_size(op, lens, news, Hq, Hkv, D, page, window, sinks):
    """Shapes of the kernel whose warps share a row, and of a warp with a row to itself."""
    c = Case(lens, news, Hq, Hkv, D, page, FP if D == 80 else BF, window, sinks, seed=32)
    check(c, run(c, op), c.reference(), op)

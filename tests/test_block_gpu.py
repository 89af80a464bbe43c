"""Norms, rotary positions and log probabilities (include/moe_block.h,
moe_kv_append_rope) against their definitions in 64 bits."""
import math

import pytest
import torch

from routed_expert_ffn_router_gb300 import _lib
from routed_expert_ffn_router_gb300 import build as libbuild
from routed_expert_ffn_router_gb300.block import Rotary, rms_norm, token_logprobs
from tests import _block_ref as ref
from tests._block_ref import within
from tests._kv_ref import Case

pytestmark = pytest.mark.gpu
BF, HF, FP, E4 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn
INF = math.inf


@pytest.fixture(scope="module", autouse=True)
def _built():
    libbuild.build()
    _lib.load()


def rnd(*shape, seed=0, dtype=FP, std=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * std).to(dtype).cuda()


# ------------------------------------------------------------------ norm
NORMS = [
    # T, H, x, residual, weight, out
    (1, 2048, FP, BF, BF, BF), (8, 2048, BF, BF, BF, BF), (3, 512, HF, HF, FP, HF), (5, 4096, BF, FP, BF, FP),
    (2, 8192, FP, FP, HF, BF), (3, 8200, BF, BF, BF, BF), (2, 16384, FP, BF, BF, HF), (700, 256, BF, BF, None, BF),
    (4, 2048, BF, None, BF, BF), (4, 2048, FP, None, None, FP), (3, 1, FP, BF, BF, BF), (3, 7, BF, BF, FP, BF),
    (5, 1023, HF, FP, BF, FP), (2, 16383, BF, BF, BF, BF), (9, 40, BF, HF, BF, HF),
]


@pytest.mark.parametrize("T,H,x,r,w,o", NORMS)
def test_norm(T, H, x, r, w, o):
    xt = rnd(T, H, seed=1, dtype=x)
    rt = None if r is None else rnd(T, H, seed=2, dtype=r, std=3.0)
    wt = None if w is None else rnd(H, seed=3, dtype=w)
    want_r, y, tol = ref.norm(xt, wt, rt, 1e-5, 0.5, o)
    got = rms_norm(xt, wt, residual=rt, eps=1e-5, weight_offset=0.5, out_dtype=o)
    assert got.dtype == o and got.shape == (T, H)
    if rt is not None:
        assert torch.equal(rt, want_r)
    within(got, y, tol, "norm")


@pytest.mark.parametrize("H,group", [(2048, 0), (2048, 128), (2048, 16), (4096, 1024), (8192, 32), (16384, 512),
                                     (100, 0), (8200, 0), (12288, 4096), (1048, 0)])
@pytest.mark.parametrize("vec", [True, False])
def test_norm_in_8_bits(H, group, vec):
    T = 5
    xt = rnd(T, H + 8, seed=1, dtype=BF)[:, 0 if vec else 1:][:, :H]  # rows on 16 bytes, or off them
    rt = rnd(T, H, seed=2, dtype=BF, std=2.0)
    xt[1] = 0
    rt[1] = 0                                     # a row of zeros
    xt[2, :H // 2] = 0
    rt[2, :H // 2] = 0                            # groups of zeros
    wt = rnd(H, seed=3, dtype=BF)
    want_r, y, tol = ref.norm(xt, wt, rt, 1e-6, 0.0, E4)
    q, s = rms_norm(xt, wt, residual=rt, eps=1e-6, out_dtype=E4, group=group)
    assert torch.equal(rt, want_r)
    n = H // group if group else 1
    assert q.dtype == E4 and s.shape == (T, n)
    top = y.reshape(T, n, -1).abs().amax(2)
    within(s, top / 448, (top / 448) * 112 * ref.F + 1e-44, "scales")
    sc = s.double().repeat_interleave(H // n, 1)
    back = q.double() * sc
    # half a step of e4m3 relative to the value, of its smallest step below the normal range
    within(back, y, tol + back.abs() * 2 ** -4 / (1 - 2 ** -4) + sc * 2 ** -10 + y.abs() * 128 * ref.F, "e4m3")
    assert (q.double().abs().reshape(T, n, -1).amax(2)[top > 0] == 448).all()


def test_norm_special_values():
    x = rnd(6, 64, dtype=FP)
    x[0] = 0
    x[1, 5] = math.nan
    x[2, 7] = INF
    x[3] *= 1e-22          # squares vanish beside eps
    x[4] *= 1e25           # squares beyond fp32
    y = rms_norm(x, eps=1e-6)
    assert (y[0] == 0).all() and torch.isnan(y[1]).all()
    assert torch.isnan(y[2, 7]) and (y[2, :7] == 0).all()
    within(y[3:4], *ref.norm(x[3:4], None, None, 1e-6, 0, FP)[1:], "small")
    assert (y[4] == 0).all()
    within(y[5:], *ref.norm(x[5:], None, None, 1e-6, 0, FP)[1:], "plain")
    z = torch.zeros(1, 64, device="cuda")
    assert torch.isnan(rms_norm(z, eps=0.0)).all()      # 0 / 0, as the formula


def test_norm_in_place_strided_and_parts():
    wide = rnd(33, 3, 256, dtype=BF)
    x = wide[:, 1]                                       # rows 768 apart
    keep = wide.clone()
    _, y, tol = ref.norm(x, None, None, 1e-6, 0, BF)
    assert rms_norm(x, out=x) is x
    within(x, y, tol, "in place")
    assert torch.equal(wide[:, 0], keep[:, 0]) and torch.equal(wide[:, 2], keep[:, 2])
    big = rnd(3, 16384, dtype=BF, seed=4)
    _, y, tol = ref.norm(big, None, None, 1e-6, 0, BF)
    within(rms_norm(big, out=big), y, tol, "in place, four groups a thread")


# ------------------------------------------------------------------ rotary positions
def rope_case(c, rot, layout, scaling, positions=None, in_place=False, max_rows=None):
    """append_rotary on a cache case, everything else of the pools untouched."""
    kv = c.cache()
    dev = c.k.device
    k_new, v_new = rnd(c.T, c.Hkv, c.D, seed=5, dtype=c.dtype), rnd(c.T, c.Hkv, c.D, seed=6, dtype=c.dtype)
    r = Rotary(rot, layout=layout, scaling=scaling)
    tok = torch.cat([torch.arange(L - n, L) for L, n in zip(c.lens_l, c.news_l)]).to(dev)
    real = tok >= 0
    pos = tok if positions is None else positions.long()
    k0, v0 = c.k.clone(), c.v.clone()
    q = c.q.clone() if in_place else c.q
    want_q, tol_q = ref.turned(c.q, pos, r.frequencies, r.gain, rot, layout)
    want_k, tol_k = ref.turned(k_new, pos, r.frequencies, r.gain, rot, layout)
    u, tiny = ref.half_step(c.dtype), ref.TINY[c.dtype]
    got = kv.append_rotary(0, q, k_new, v_new, r, slots=c.slots, row_start=c.row_start, positions=positions,
                           q_out=q if in_place else None)
    assert kv.status() == (_lib.MOE_OK, 0)
    assert (got is q) == in_place
    within(got[real], want_q[real], (tol_q + u * want_q.abs() + tiny)[real], "q")
    assert torch.equal(got[~real], c.q[~real])
    at = 0
    for s, L, n in zip(c.slots.tolist(), c.lens_l, c.news_l):
        for i in range(n):
            t = L - n + i
            if t >= 0:
                pg, j = int(c.table[s, t // c.page]), t % c.page
                within(c.k[0, pg, :, j], want_k[at], tol_k[at] + u * want_k[at].abs() + tiny, "k")
                assert torch.equal(c.v[0, pg, :, j], v_new[at])
                k0[0, pg, :, j], v0[0, pg, :, j] = c.k[0, pg, :, j], c.v[0, pg, :, j]
            at += 1
    same = lambda a, b: torch.equal(a.view(torch.int16), b.view(torch.int16))  # noqa: E731
    assert same(c.k, k0) and same(c.v, v0)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("D,rot,dtype", [(128, 128, BF), (128, 64, HF), (64, 64, BF), (80, 80, BF), (80, 40, HF),
                                         (256, 256, BF), (8, 2, BF), (128, 6, BF), (72, 70, HF), (128, 112, BF)])
def test_rotary(D, rot, layout, dtype):
    c = Case([40, 1, 133], [17, 1, 60], 8, 2, D, 16, dtype, seed=1)
    rope_case(c, rot, layout, None)


@pytest.mark.parametrize("scaling", [dict(kind="linear", factor=4), dict(kind="ntk", factor=8),
                                     dict(kind="yarn", factor=4, original=8192),
                                     dict(kind="bands", factor=8, original=8192, low=1, high=4)])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotary_scaled_far_positions(scaling, layout):
    c = Case([131057, 20000], [3, 2], 5, 5, 64, 64, BF, seed=2, window=16)
    rope_case(c, 64, layout, scaling, in_place=True)


def test_rotary_given_positions_and_rows_before_the_first_token():
    c = Case([2, 9], [4, 4], 4, 1, 64, 8, BF, seed=3)  # rows of tokens -2 and -1
    rope_case(c, 64, "half", None)
    c = Case([30, 9], [4, 4], 4, 1, 64, 8, BF, seed=3)
    p = torch.tensor([0, 7, 2 ** 31 - 1, -5, 1000003, 12, 12, 1], dtype=torch.int32).cuda()
    rope_case(c, 64, "interleaved", None, positions=p)


def test_rotary_bad_slots_pages_and_rows_behind():
    c = Case([30, 20], [2, 2], 4, 2, 64, 8, BF, seed=4)
    kv, r = c.cache(), Rotary(64)
    slots = c.slots.clone()
    slots[0] = 77
    k = rnd(6, 2, 64, dtype=BF)
    k0 = c.k.clone()
    q = rnd(6, 4, 64, dtype=BF, seed=9)
    out = torch.full_like(q, 7.0)
    start = torch.tensor([0, 2, 4], dtype=torch.int32).cuda()
    kv.append_rotary(0, q, k, k, r, slots=slots, row_start=start, q_out=out)
    assert kv.status()[1] == 2
    assert torch.equal(out[:2], q[:2])                   # no tokens: copied
    assert (out[4:] == 7).all()                          # behind the last sequence
    assert not torch.equal(out[2:4], q[2:4])
    kv.clear_status()
    c.table[int(c.slots[1]), 2] = 1 << 20                # the new tokens' page
    k1 = c.k.clone()
    kv.append_rotary(0, q[:2], k[:2], k[:2], r, slots=c.slots[1:].contiguous(), row_start=start[:2].contiguous(), q_out=out[:2])
    assert kv.status()[1] == 2
    assert torch.equal(c.k.view(torch.int16), k1.view(torch.int16)) and not torch.equal(out[:2], q[:2])
    assert not torch.equal(k0.view(torch.int16), k1.view(torch.int16))


def test_rotary_then_attention_goes_by_distance():
    """Scores of turned queries and keys depend on the distance alone: the same rows at
    other positions give the same attention up to roundings."""
    outs = []
    for shift in (0, 1000):
        c = Case([50], [50], 4, 2, 128, 16, HF, seed=6)
        kv, r = c.cache(), Rotary(128)
        k, v = rnd(50, 2, 128, dtype=HF, seed=7), rnd(50, 2, 128, dtype=HF, seed=8)
        pos = (torch.arange(50) + shift).to(torch.int32).cuda()
        q = kv.append_rotary(0, c.q, k, v, r, slots=c.slots, row_start=c.row_start, positions=pos)
        outs.append(kv.chunk(0, q, slots=c.slots, row_start=c.row_start).double())
        assert kv.status() == (_lib.MOE_OK, 0)
    # scores: 128 products of two values rounded once (2^-11 each) of size 1.5, at D^-0.5; outputs of size 1
    assert (outs[0] - outs[1]).abs().max() < 4 * 2 ** -11 * 1.5 * 128 ** 0.5


# ------------------------------------------------------------------ log probabilities
def check_logprobs(z, tokens, top, temperature=1.0):
    want, tol = ref.logprobs(z, tokens, top, temperature)
    got = token_logprobs(z, tokens, top=top, temperature=temperature)
    assert set(got) == set(want)
    for n in want:
        if n in ("rank", "top_ids"):
            assert torch.equal(got[n], want[n]), n
        else:
            within(got[n], want[n], tol[n], n)


@pytest.mark.parametrize("T,V,top,dtype,pad", [
    (1, 32000, 5, FP, 0), (3, 50257, 20, BF, 0), (2, 1, 1, BF, 0), (5, 2, 2, HF, 0), (7, 33, 32, BF, 0), (4, 1000, 0, BF, 24),
    (300, 777, 1, HF, 1), (64, 4097, 32, FP, 3), (1, 200003, 32, BF, 0), (2, 131072, 8, HF, 8), (160, 9000, 3, BF, 7),
])
@pytest.mark.parametrize("temperature", [1.0, 0.6])
def test_logprobs(T, V, top, dtype, pad, temperature):
    z = rnd(T, V + pad, seed=T, dtype=dtype, std=3.0)[:, pad // 2:pad // 2 + V]
    tok = torch.randint(0, V, (T,), generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()
    tok[0] = z[0].argmax()
    tok[-1] = V - 1
    check_logprobs(z, tok, top, temperature)


@pytest.mark.parametrize("dtype", [FP, BF, HF])
@pytest.mark.parametrize("V", [40, 5000, 70001])
def test_logprobs_ties_order_and_masks(V, dtype):
    T = 8
    z = rnd(T, V, seed=3, dtype=dtype, std=2.0)
    low = torch.finfo(dtype).min
    z[0] = 1.25                                     # all equal: the lowest ids
    z[1] = torch.arange(V).to(dtype).cuda()         # ever larger (equal in 16 bits for long)
    z[2] = -torch.arange(V).float().cuda().to(dtype)
    z[3] = low                                      # nothing but the lowest value: uniform
    z[4, 1:] = -INF                                 # one token left
    z[5, ::2] = low
    z[6] = torch.where(torch.arange(V).cuda() % 7 == 0, z[6], torch.full_like(z[6], -INF))
    z[7] = (torch.arange(V) % 2).float().cuda() * -0.0     # 0 and -0 are equal
    if dtype is not FP:
        z[2].clamp_(min=-30000)
        z[1].clamp_(max=30000)
    tok = torch.tensor([V // 2, V - 1, 0, V - 1, 0, 1, 1, V - 1], dtype=torch.int32).cuda()
    check_logprobs(z, tok, 32)


def test_logprobs_special_rows():
    V = 3000
    z = rnd(6, V, dtype=FP)
    z[0] = -INF
    z[1, 17] = math.nan
    z[2, 2999] = INF
    z[3, 0] = -INF
    tok = torch.tensor([4, 17, 3, 0, -1, V], dtype=torch.int32).cuda()
    r = token_logprobs(z, tok, top=4)
    assert r["logprob"][0] == -INF and r["entropy"][0] == 0 and r["rank"][0] == 4
    assert r["top_ids"][0].tolist() == [0, 1, 2, 3] and (r["top_logprobs"][0] == -INF).all()
    for i in (1, 2):
        assert torch.isnan(r["logprob"][i]) and torch.isnan(r["entropy"][i]) and torch.isnan(r["top_logprobs"][i]).all()
    assert r["top_ids"][1].tolist() == torch.sort(z[1].nan_to_num(-INF), descending=True, stable=True)[1][:4].tolist()
    assert r["rank"][1] == V - 1                    # with -inf, behind all
    assert r["top_ids"][2, 0] == 2999
    assert r["logprob"][3] == -INF and r["rank"][3] == V - 1
    assert r["logprob"][4:].tolist() == [0, 0] and r["rank"][4:].tolist() == [-1, -1]
    want, tol = ref.logprobs(z[4:], None, 4, 1.0)
    within(r["entropy"][4:], want["entropy"], tol["entropy"], "entropy of padded rows")


def test_logprobs_without_tokens_and_into_given_tensors():
    z = rnd(3, 600, dtype=BF)
    assert set(token_logprobs(z)) == {"entropy"}
    out = {"entropy": torch.empty(3, device="cuda"), "top_ids": torch.empty(3, 2, dtype=torch.int32, device="cuda"),
           "top_logprobs": torch.empty(3, 2, device="cuda")}
    r = token_logprobs(z, top=2, out=out)
    assert all(r[n] is out[n] for n in out) and torch.equal(r["top_ids"][:, 0].long(), z.argmax(1))
    assert _lib.moe_last_launch_count() == 1


def test_no_rows():
    e = torch.empty(0, 64, device="cuda")
    assert rms_norm(e).shape == (0, 64)
    assert token_logprobs(e, torch.empty(0, dtype=torch.int32, device="cuda"), top=3)["top_ids"].shape == (0, 3)


# ------------------------------------------------------------------ streams and graphs
def test_on_another_stream_and_in_graphs():
    x, r, w = rnd(9, 2048), rnd(9, 2048, seed=1, dtype=BF), rnd(2048, dtype=BF)
    z, tok = rnd(9, 5003, dtype=BF), torch.arange(9, dtype=torch.int32).cuda()
    want_y = rms_norm(x, w, residual=r.clone())
    want = token_logprobs(z, tok, top=5)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for stream in (s, s.cuda_stream):
        res = r.clone()
        s.wait_stream(torch.cuda.current_stream())
        y = rms_norm(x, w, residual=res, stream=stream)
        got = token_logprobs(z, tok, top=5, stream=stream)
        s.synchronize()
        assert torch.equal(y, want_y) and all(torch.equal(got[n], want[n]) for n in want)
    res = r.clone()
    y, outs = torch.empty_like(r), [{n: torch.empty_like(t) for n, t in want.items()} for _ in range(2)]
    graphs = []
    for out in outs:  # two graphs of the same calls
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            rms_norm(x, w, residual=res, out=y)
            token_logprobs(z, tok, top=5, out=out)
        graphs.append(g)
    res.copy_(r)
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want_y)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    z.copy_(rnd(9, 5003, dtype=BF, seed=5))
    want = token_logprobs(z, tok, top=5)
    torch.cuda.synchronize()
    for i, st in enumerate((s1, s2)):
        with torch.cuda.stream(st):
            if i == 0:
                graphs[0].replay()
            else:
                token_logprobs(z, tok, top=5, out=outs[1])
    torch.cuda.synchronize()
    for out in outs:
        assert all(torch.equal(out[n], want[n]) for n in want)


def test_logprobs_of_rows_beyond_what_fits_at_once():
    """Rows for several turns of the CTAs that fit on the GPU."""
    T, V = 700, 33001
    z = torch.randn(T, V, generator=torch.Generator(device="cuda").manual_seed(8), device="cuda").bfloat16()
    tok = torch.arange(T, dtype=torch.int32, device="cuda")
    check_logprobs(z, tok, 3)
    first = token_logprobs(z[:50], tok[:50], top=3)
    assert torch.equal(first["top_ids"], token_logprobs(z, tok, top=3)["top_ids"][:50])


@pytest.mark.parametrize("T,V,dtype", [(1, 32000, torch.float32), (6, 50257, torch.bfloat16), (700, 9001, torch.float16)])
def test_logprobs_of_a_token_with_nearly_all(T, V, dtype):
    """Logarithm and entropy of a row in which one token (rarely two equal ones) has all but
    e^-6 to e^-20: right relative to themselves. The rest, sum e^d: each term's argument is
    off by 3 F |d| (difference, factor, product), its exponential by 4 F, and it goes
    through at most V / 256 + 60 additions of a relative F; ln(1 + rest), the entropy's
    quotient, products and sum: 16 F."""
    g = torch.Generator(device="cuda").manual_seed(3)
    z = torch.randn(T, V, generator=g, device="cuda")
    at = torch.randint(0, V, (T,), generator=g, device="cuda")
    z.scatter_(1, at[:, None], (math.log(V) + 6 + 14 * torch.rand(T, 1, generator=g, device="cuda")))
    z = z.to(dtype)
    tok = z.argmax(1).int()
    got = token_logprobs(z, tok, top=2)
    d = z.double() - z.double().amax(1, keepdim=True)
    d.scatter_(1, tok.long()[:, None], -INF)
    e = torch.exp(d)
    rest, far = e.sum(1), torch.where(e > 0, -d, torch.zeros_like(d)).amax(1)
    want = -torch.log1p(rest)
    ent = -want - torch.where(e > 0, e * d, torch.zeros_like(d)).sum(1) / (1 + rest)
    part = (V / 256 + 60 + 3 * far + 4 + 16) * ref.F
    within(got["logprob"], want, part * want.abs(), "logprob")
    within(got["top_logprobs"][:, 0], want, part * want.abs(), "top")
    within(got["entropy"], ent, (part + 3 * ref.F) * ent, "entropy")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_logprobs_order_of_subnormal_logits(dtype):
    """Logits below the type's normal range are in their order too, and either zero ties."""
    g = torch.Generator(device="cuda").manual_seed(9)
    T, V = 12, 20011
    step = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    z = (torch.randint(-60, 61, (T, V), generator=g, device="cuda").double() * step).to(dtype)
    z[:, ::7] = -0.0
    tok = torch.randint(0, V, (T,), generator=g, device="cuda").int()
    got = token_logprobs(z, tok, top=8)
    order = torch.sort(z.double(), dim=1, descending=True, stable=True)[1]
    assert torch.equal(got["rank"], (order == tok[:, None]).int().argmax(1).int())
    assert torch.equal(got["top_ids"], order[:, :8].int())

"""Attention over the paged cache at the edges of its arguments, against the
64-bit definition: very large windows and first-token counts, rows before the
first token next to values that are not finite, probabilities far below the
largest."""
import math

import pytest
import torch

from routed_expert_ffn_router_gb300 import _lib
from routed_expert_ffn_router_gb300 import build as libbuild
from tests._kv_ref import Case, check

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16
MOST = 2 ** 31 - 1


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


@pytest.mark.parametrize("D,page", [(64, 16), (128, 64), (80, 24)])
@pytest.mark.parametrize("op", ["decode", "chunk"])
@pytest.mark.parametrize("window,sinks", [(200, MOST), (200, MOST - 127), (1, MOST), (MOST, 0), (MOST, MOST), (MOST, 5)])
def test_windows_and_first_tokens_without_bound(op, D, page, window, sinks):
    n = (2, 2) if op == "decode" else (300, 17)
    c = Case([1500, 40], n, 8, 2, D, page, BF, window, sinks, seed=41)
    check(c, run(c, op), c.reference(), op)


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("lens,n,Hq,Hkv,D", [([1, 2, 0], 3, 4, 2, 128), ([1, 2, 3, 20], 3, 8, 2, 64),
                                             ([5, 15, 16], 16, 4, 2, 128), ([1], 2, 4, 2, 80)])
def test_rows_before_the_first_token_next_to_values_that_are_not_finite(bad, lens, n, Hq, Hkv, D):
    # the rows of a window that are no tokens see nothing, whatever the first token holds
    c = Case(lens, [n] * len(lens), Hq, Hkv, D, 16, BF, 0, 0, seed=42)
    for b, s in enumerate(c.slots.tolist()):
        if lens[b]:
            c.v[0, int(c.table[s, 0]), :, 0] = bad
    check(c, run(c, "decode"), c.reference(), "not finite")


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("op,n,D", [("decode", 1, 128), ("decode", 4, 64), ("chunk", 1, 64), ("chunk", 700, 128),
                                    ("chunk", 700, 64)])
def test_probabilities_far_below_the_largest(dtype, op, n, D):
    """Every sixteenth key has score 0 and the value 0, the others a score of about
    -25.5 ln 2 and a large value: only the small probabilities reach the result. A
    probability in fp16 has a fixed step below the normal range: with the largest lifted
    to 2^7, half of it is 2^-32 of the largest probability, for each key."""
    c = Case([1800], [n], 8, 2, D, 16, dtype, 0, 0, seed=43, poison=False)
    c.q.zero_()
    c.q[..., 0] = 4.0
    c.k.zero_()
    c.k[..., 0] = -17.675 / 4
    c.k[..., 0::16, :] = 0.0
    c.v[:] = 1000.0 + 10 * torch.randn(c.v.shape, device="cuda").to(dtype)
    c.v[..., 0::16, :] = 0.0
    ro, rl, to, tl = c.reference(scale=1.0)
    if dtype == FP:
        to = to + 1.05 * 16 * 2.0 ** -32 * float(c.v.max())   # at most 16 keys for each of the largest ones
    assert float(ro.min()) > 20 * float(to.max())
    check(c, run(c, op, scale=1.0), (ro, rl, to, tl), op)

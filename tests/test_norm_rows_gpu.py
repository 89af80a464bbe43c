"""Norms of more rows than CTAs fit on the GPU (include/moe_block.h): a CTA goes on to
further rows, whose loads are ahead of its stores and whose sums, scales and
maxima take the place of the rows' before. At least three turns each and a last
one that is not full; neighbours of a CTA differ by powers of two in size, so that
a sum or a scale of another row shows."""
import pytest
import torch

from routed_expert_ffn_router_gb300 import _lib
from routed_expert_ffn_router_gb300 import build as libbuild
from routed_expert_ffn_router_gb300.block import rms_norm
from tests import _block_ref as ref
from tests._block_ref import within

pytestmark = pytest.mark.gpu
BF, HF, FP, E4 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _built():
    libbuild.build()
    _lib.load()


def rows(T, H, seed, dtype):
    """Normal values times 2^-7 .. 2^7 by the row: rows a grid apart differ."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, H, generator=g, device="cuda")
    return (x * torch.exp2((torch.arange(T, device="cuda") * 7 // 5 % 15 - 7).float())[:, None]).to(dtype)


# at most 6 CTAs per SM up to 2,048 columns, 3 up to 4,096, then 1
@pytest.mark.parametrize("T,H,x,r,w,o", [
    (2741, 256, BF, BF, BF, BF), (3001, 64, BF, BF, None, HF), (2801, 1000, FP, BF, BF, BF), (2745, 2048, FP, FP, FP, FP),
    (1403, 4096, HF, HF, BF, HF), (1403, 3080, FP, BF, BF, BF), (1403, 4096, BF, None, BF, BF), (477, 8192, BF, BF, BF, BF),
    (477, 5120, FP, HF, FP, BF), (477, 16384, BF, BF, BF, BF), (477, 16384, FP, FP, BF, FP), (477, 10248, BF, BF, BF, HF),
])
def test_norm(T, H, x, r, w, o):
    xt, rt = rows(T, H, 1, x), None if r is None else rows(T, H, 2, r)
    wt = None if w is None else rows(1, H, 3, w)[0] * 2 ** 7
    want_r, y, tol = ref.norm(xt, wt, rt, 1e-5, 0.25, o)
    got = rms_norm(xt, wt, residual=rt, eps=1e-5, weight_offset=0.25, out_dtype=o)
    assert rt is None or torch.equal(rt, want_r)
    within(got, y, tol, "norm")


@pytest.mark.parametrize("T,H,group,x", [
    (2741, 2048, 0, BF), (2741, 2048, 128, BF), (2741, 2048, 1024, BF), (3001, 64, 16, BF), (3001, 512, 512, FP), (2745, 1048, 0, FP),
    (1403, 4096, 0, FP), (1403, 4096, 128, BF), (1403, 4096, 1024, FP), (1403, 4096, 4096, BF), (477, 8192, 0, BF), (477, 6144, 2048, BF),
    (477, 16384, 0, BF), (477, 16384, 256, FP), (477, 16384, 512, BF), (477, 16384, 8192, BF),
])
def test_norm_in_8_bits(T, H, group, x):
    xt, rt = rows(T, H, 1, x), rows(T, H, 2, BF)
    for t in range(5, T, 13):                     # rows of zeros among the others
        xt[t], rt[t] = 0, 0
    wt = rows(1, H, 3, BF)[0] * 2 ** 7
    want_r, y, tol = ref.norm(xt, wt, rt, 1e-6, 0.0, E4)
    q, s = rms_norm(xt, wt, residual=rt, eps=1e-6, out_dtype=E4, group=group)
    assert torch.equal(rt, want_r)
    n = H // group if group else 1
    top = y.reshape(T, n, -1).abs().amax(2)
    within(s, top / 448, (top / 448) * 112 * ref.F + 1e-44, "scales")
    sc = s.double().repeat_interleave(H // n, 1)
    back = q.double() * sc
    # half a step of e4m3 relative to the value, of its smallest step below the normal range
    within(back, y, tol + back.abs() * 2 ** -4 / (1 - 2 ** -4) + sc * 2 ** -10 + y.abs() * 128 * ref.F, "e4m3")
    assert (q.double().abs().reshape(T, n, -1).amax(2)[top > 0] == 448).all()
    assert (s[top == 0] == 0).all() and (q.double()[y == 0] == 0).all()


@pytest.mark.parametrize("T,H,dtype", [(2741, 2048, BF), (1403, 4096, HF), (477, 16384, BF), (2741, 1024, FP)])
def test_norm_in_place_beside_a_residual(T, H, dtype):
    xt, rt = rows(T, H, 1, dtype), rows(T, H, 2, BF)
    want_r, y, tol = ref.norm(xt, None, rt, 1e-6, 0.0, dtype)
    assert rms_norm(xt, residual=rt, out=xt) is xt
    assert torch.equal(rt, want_r)
    within(xt, y, tol, "in place")


def test_norm_of_strided_rows():
    wide, res = rows(2741, 3 * 512, 1, BF), rows(2741, 2 * 512, 2, BF)
    keep_w, keep_r = wide.clone(), res.clone()
    x, r = wide[:, 512:1024], res[:, 512:]
    want_r, y, tol = ref.norm(x, None, r, 1e-6, 0.0, BF)
    out = torch.full((2741, 4 * 512), 3.0, dtype=BF, device="cuda")
    rms_norm(x, residual=r, out=out[:, 1024:1536])
    within(out[:, 1024:1536], y, tol, "strided")
    assert torch.equal(r, want_r) and torch.equal(wide, keep_w) and torch.equal(res[:, :512], keep_r[:, :512])
    assert (out[:, :1024] == 3).all() and (out[:, 1536:] == 3).all()

"""Linear attention of prompt chunks whose sequences are divided over the CTAs of a
cluster (include/moe_block.h): few heads and long prompts."""
import pytest
import torch

from routed_expert_ffn_router_gb300 import build as libbuild
from routed_expert_ffn_router_gb300 import _lib
from tests import _linear_ref
from tests._block_ref import within
from tests.test_linear_gpu import Inputs, check

gpu = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _built():
    libbuild.build()
    _lib.load()


@gpu
@pytest.mark.parametrize("dtype", [BF, HF])
def test_first_part_reads_the_initial_state_before_the_last_writes_the_final_one(dtype):
    """Two CTAs per sequence and head; the short sequence has a block in each, so its end is
    written soonest after its start is read. With memory kept busy from another stream
    every call gives the same bits."""
    i = Inputs([900, 129], 16, 32, 128, 128, dtype, seed=21)
    layer = i.layer()
    want = layer.chunk(i.q, i.k, i.v, i.g, slots=i.slots, row_start=i.start)
    check(i, layer, want, 128 ** -0.5, True)
    end, other, o = layer.state.clone(), torch.cuda.Stream(), torch.empty_like(want)
    a = torch.zeros(1 << 28, dtype=torch.uint8, device="cuda")
    b = torch.empty_like(a)
    torch.cuda.synchronize()
    for _ in range(40):
        layer.state.copy_(i.state)
        with torch.cuda.stream(other):
            b.copy_(a)
        layer.chunk(i.q, i.k, i.v, i.g, slots=i.slots, row_start=i.start, out=o)
        assert torch.equal(o, want) and torch.equal(layer.state, end)
    assert layer.status() == 0


# Hk, Hv, Dk, Dv, dtype: head sizes alike and not, both types
SHAPES = [(2, 4, 128, 128, HF), (4, 8, 128, 128, BF), (1, 2, 64, 64, HF), (1, 2, 64, 64, BF), (2, 2, 64, 128, BF), (1, 3, 64, 128, HF),
          (2, 2, 128, 64, BF), (1, 1, 128, 64, HF)]
# rows: eight CTAs per sequence and head (mean of 16 blocks or more), four, two with sequences
# that end in the first CTA's part, in the second's, or have no rows
NEWS = [[2177], [1100], [700, 130, 1500, 0, 600]]


@gpu
@pytest.mark.parametrize("decay", ["mixed", "none", "strong", "resets"])
@pytest.mark.parametrize("Hk,Hv,Dk,Dv,dtype", SHAPES)
@pytest.mark.parametrize("news", NEWS)
def test_divided_sequences(news, Hk, Hv, Dk, Dv, dtype, decay):
    i = Inputs(news, Hk, Hv, Dk, Dv, dtype, seed=Hv + len(news), decay=decay)
    layer = i.layer()
    check(i, layer, layer.chunk(i.q, i.k, i.v, i.g, slots=i.slots, row_start=i.start), Dk ** -0.5, True)


class Sparse(Inputs):
    """Keys at two tokens of each block of 128 only, in different 16s; decays between none and
    e^-4 a block, so that what the CTAs of a cluster hand on is neither all nor nothing."""

    def __init__(self, news, Hk, Hv, Dk, Dv, dtype, seed, decay):
        super().__init__(news, Hk, Hv, Dk, Dv, dtype, seed=seed, decay=decay, state=seed % 2 == 0)
        if decay == "mixed":
            self.g *= 0.02
        r = torch.Generator().manual_seed(seed)
        keep = torch.zeros(self.T, dtype=torch.bool)
        for _, r0, n in self.spans():
            for b in range(0, n, 128):
                for at in (torch.randperm(8, generator=r)[:2] * 16 + torch.randint(0, 16, (2,), generator=r)).tolist():
                    if b + at < n:
                        keep[r0 + b + at] = True
        self.k *= 8
        self.k[~keep.to(self.k.device)] = 0


@gpu
@pytest.mark.parametrize("decay", ["mixed", "none", "strong", "resets"])
@pytest.mark.parametrize("Hk,Hv,Dk,Dv,dtype", SHAPES)
@pytest.mark.parametrize("news", [[1100], [700, 130, 1500, 0, 600], [300, 20]])
def test_state_within_its_own_roundings(news, Hk, Hv, Dk, Dv, dtype, decay):
    i = Sparse(news, Hk, Hv, Dk, Dv, dtype, seed=Hv + len(news) + Dk, decay=decay)
    layer = i.layer()
    layer.chunk(i.q, i.k, i.v, i.g, slots=i.slots, row_start=i.start)
    want, tol = _linear_ref.state(i.k, i.v, i.g, i.state, i.spans(), 2)
    assert layer.status() == 0
    within(layer.state, want, tol, "state")


def test_the_bound_shows_keys_of_two_values(monkeypatch):
    """Two values of bf16 for a decayed key, as the oracle plants them, are outside the bound of
    three. No GPU needed."""
    monkeypatch.setattr(torch.Tensor, "cuda", lambda self: self)
    i = Sparse([300, 20], 1, 2, 64, 64, BF, seed=3, decay="mixed")
    want, tol = _linear_ref.state(i.k, i.v, i.g, i.state, i.spans(), 2)
    off, _ = _linear_ref.state(i.k, i.v, i.g, i.state, i.spans(), 2, two_values=True)
    assert ((off - want).abs() > tol)[i.slots.long()].float().mean() > 0.02

"""Linear attention of prompt chunks whose sequences are divided over the CTAs of a
cluster (include/moe_block.h): few heads and long prompts."""
import pytest
import torch

from routed_expert_ffn_router_gb300 import build as libbuild
from routed_expert_ffn_router_gb300 import _lib
from tests.test_linear_gpu import Inputs, check

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _built():
    libbuild.build()
    _lib.load()


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

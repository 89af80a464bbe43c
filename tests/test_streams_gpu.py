"""Calls on a stream that is not the current one: the tensors that a wrapper
allocates for its results belong to the stream that writes them, whatever the
current stream still has queued for the memory it would hand out."""
import pytest
import torch

from routed_expert_ffn_router_gb300 import _lib
from routed_expert_ffn_router_gb300 import build as libbuild
from tests._kv_ref import Case

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
BUSY = 200_000_000  # cycles, about a tenth of a second


@pytest.fixture(scope="module", autouse=True)
def _built():
    libbuild.build()
    _lib.load()


def left_behind(*shapes):
    """The current stream is busy, and then fills freed blocks of these sizes."""
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    blocks = [torch.empty(s, dtype=dt, device="cuda") for s, dt in shapes]
    torch.cuda._sleep(BUSY)
    for b in blocks:
        b.fill_(7)


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("op", ["decode", "chunk"])
def test_attention_results_on_another_stream(op, raw):
    n = 2 if op == "decode" else 100
    c = Case([300, 200], [n, n], 8, 2, 128, 16, BF, 0, 0, seed=51)
    kv = c.cache()
    rows = {} if op == "decode" else dict(row_start=c.row_start)
    call = getattr(kv, op)
    want = call(0, c.q, slots=c.slots, want_lse=True, **rows)
    s = torch.cuda.Stream()
    left_behind((want[0].shape, BF), (want[1].shape, torch.float32))
    got = call(0, c.q, slots=c.slots, want_lse=True, stream=s.cuda_stream if raw else s, **rows)
    s.synchronize()
    torch.cuda.synchronize()
    assert kv.status() == (_lib.MOE_OK, 0)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])

"""Calls on a stream that is not the current one: the tensors that a wrapper
allocates for its results belong to the stream that writes them, whatever the
current stream still has queued for the memory it would hand out."""
import pytest
import torch

from routed_expert_ffn_router_gb300 import _lib, synth
from routed_expert_ffn_router_gb300 import build as libbuild
from routed_expert_ffn_router_gb300.layer import MoeLayer
from routed_expert_ffn_router_gb300.mailbox import Mailbox
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


@pytest.mark.parametrize("raw", [False, True])
def test_layer_results_on_another_stream(raw):
    cfg = synth.MoeConfig("streams", H=512, I=256, E=32, k=4, T=16, zipf_s=1.0, resident_frac=0.5)
    inp = synth.make_layer(cfg, 5, device="cuda")
    lay = MoeLayer(inp, T_max=cfg.T)
    logits, xs = synth.draw_windows(inp, 1, seed=9)
    want = lay.forward(logits[0], xs[0])
    assert int(want["n_miss"]) > 0
    s = torch.cuda.Stream()
    left_behind(*[(t.shape, t.dtype) for t in want.values()])
    got = lay.forward(logits[0], xs[0], stream=s.cuda_stream if raw else s)
    again = lay.expert_ffn(xs[0], want["ids"], want["w"], stream=s.cuda_stream if raw else s)
    s.synchronize()
    torch.cuda.synchronize()
    assert lay.status()[0] == _lib.MOE_OK
    n = int(want["n_miss"])
    for k in ("y", "ids", "w", "n_miss"):
        assert torch.equal(got[k], want[k]), k
    assert torch.equal(got["miss_ids"][:n], want["miss_ids"][:n])
    assert torch.equal(again["y"], want["y"]) and torch.equal(again["n_miss"], want["n_miss"])


@pytest.mark.parametrize("raw", [False, True])
def test_mailbox_window_on_another_stream(raw):
    cfg = synth.MoeConfig("mbstreams", H=1024, I=512, E=64, k=8, T=16, zipf_s=1.2)
    store = synth.make_layer(cfg, 5)
    smt, S = synth.random_slot_map(cfg.E, 0.6, seed=2)
    pool = synth.make_layer(cfg, 5)
    keep = (smt >= 0).nonzero().flatten()
    for name in ("gate_q", "gate_s", "up_q", "up_s", "down_q", "down_s"):
        setattr(pool, name, getattr(pool, name)[keep].contiguous())
    pool.S, pool.slot_map = S, smt
    pool = pool.to(torch.device("cuda", 0))
    lay = MoeLayer(pool, T_max=cfg.T)
    mb = Mailbox(store, n_threads=4)
    want = mb.forward(lay, pool.logits, pool.x, pool.slot_map)
    n = len(want["mailbox_pairs"])
    assert n > 0
    s = torch.cuda.Stream()
    left_behind(((n, cfg.H), torch.float32), ((n,), torch.int32), (want["y"].shape, torch.float32))
    got = mb.forward(lay, pool.logits, pool.x, pool.slot_map, stream=s.cuda_stream if raw else s)
    s.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(got["y"], want["y"])
    mb.close()

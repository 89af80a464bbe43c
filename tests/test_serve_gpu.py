"""The serving example: prompts, branches, decode steps and a compaction through
the whole stack, with every attention call held against the 64-bit definition
on the cache's contents at that moment."""
import importlib.util
import os

import pytest
import torch

from routed_expert_ffn_router_gb300.paged import PagedKV
from tests._kv_ref import Case, check

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def serve():
    from routed_expert_ffn_router_gb300 import build
    build.build()
    spec = importlib.util.spec_from_file_location("serve_example", os.path.join(ROOT, "examples", "serve.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


class Checked(PagedKV):
    """Every attention call against the definition."""
    calls = 0

    def _attend(self, fn, layer, q, slots, row_start, scale, window, sinks, want_lse, out, lse, stream):
        o, l = super()._attend(fn, layer, q, slots, row_start, scale, window, sinks, True, out, lse, stream)
        c = Case.__new__(Case)
        c.T, c.Hq, c.Hkv, c.D, c.page, c.dtype = q.shape[0], self.Hq, self.Hkv, self.D, self.desc.page_size, self.dtype
        c.window, c.sinks, c.dev = window, sinks, self.device
        c.k, c.v, c.table, c.slots, c.q = self.k, self.v, self.table, slots, q
        c.lens_l = self.lens[slots.long()].tolist()
        start = list(range(c.T + 1)) if row_start is None else row_start.tolist()
        c.row_start = torch.tensor(start)
        c.news_l = [b - a for a, b in zip(start, start[1:])]
        check(c, (o, l), c.reference(layer))
        Checked.calls += 1
        return (o, l) if want_lse else o


PROMPTS = [[(7 * i + 3) % 64 for i in range(n)] for n in (33, 1, 16, 50)]


@pytest.mark.parametrize("window,sinks", [(0, 0), (24, 3)])
def test_every_attention_call_of_a_session(serve, window, sinks):
    model = serve.Decoder(n_layers=2, vocab=64, window=window, sinks=sinks, T_max=128)
    Checked.calls = 0
    kv = model.cache(n_pages=64, page_size=16, n_slots=12, max_tokens=80, cls=Checked)
    kv.v.fill_(float("nan"))  # a place that nothing was written to must not be read
    kv.k.fill_(float("nan"))
    tokens, logits = serve.serve(model, kv, PROMPTS, branches=2, steps=6)
    assert Checked.calls == 2 * (1 + 6)
    assert torch.isfinite(logits).all() and kv.status() == (0, 0) and all(s == (0, 0) for s in model.status())
    assert kv.lens.tolist() == [0] * 4 + [n + 6 for n in (33, 33, 1, 1, 16, 16, 50, 50)]
    # the pages in use: each prompt's full pages once, and each branch's own
    own = sum(2 * (-(-(n + 6) // 16) - n // 16) + n // 16 for n in (33, 1, 16, 50))
    assert 64 - int(kv.n_free) == own


def test_compaction_changes_no_result(serve):
    """Decode attention's result does not depend on where the pages lie: with and
    without a compaction between the steps, the same bits."""
    model = serve.Decoder(n_layers=2, vocab=64, T_max=128)
    got = []
    for compact in (False, True):
        kv = model.cache(n_pages=64, page_size=16, n_slots=12, max_tokens=80)
        got.append(serve.serve(model, kv, PROMPTS, branches=2, steps=8, compact=compact))
        assert kv.status() == (0, 0)
        if compact:  # the live pages were the lowest ones; growth took the next
            assert sorted((kv.refs > 0).nonzero()[:, 0].tolist()) == list(range(64 - int(kv.n_free)))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


def test_example_command(serve, capsys, monkeypatch):
    monkeypatch.setattr("sys.argv", ["serve.py", "--steps", "4", "--branches", "2"])
    serve.main()
    out = capsys.readouterr().out
    assert "3 prompts, 6 branches, 4 steps" in out and out.count("branch ") == 6

"""The hybrid decoder of examples/serve.py: norms, rotary positions, linear
attention and log probabilities together with the cache and the experts, every
call of a session held against its definition."""
import importlib.util
import os

import pytest
import torch

from routed_expert_ffn_router_gb300.linear import LinearAttention
from routed_expert_ffn_router_gb300.paged import PagedKV
from tests import _block_ref as ref
from tests._block_ref import within

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROMPTS = [[(7 * i + 3) % 64 for i in range(n)] for n in (133, 1, 16, 50)]


@pytest.fixture(scope="module")
def serve():
    from routed_expert_ffn_router_gb300 import build
    build.build()
    spec = importlib.util.spec_from_file_location("serve_hybrid", os.path.join(ROOT, "examples", "serve.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def run(serve, steps=6, compact=True, cls=PagedKV):
    model = serve.HybridDecoder(12, n_layers=4, vocab=64, T_max=256)
    kv = model.cache(n_pages=64, page_size=16, n_slots=12, max_tokens=160, cls=cls)
    scores = []
    tokens, logits = serve.serve(model, kv, PROMPTS, branches=2, steps=steps, compact=compact, session=serve.HybridSession,
                                 scores=scores)
    assert torch.isfinite(logits).all() and kv.status() == (0, 0) and all(s == (0, 0) for s in model.status())
    assert all(l.status() == 0 for l in model.linear.values())
    return tokens, logits, scores, model


class Checked(PagedKV):
    calls = 0

    def append_rotary(self, layer, q, k, v, rotary, slots=None, row_start=None):
        got = super().append_rotary(layer, q, k, v, rotary, slots=slots, row_start=row_start)
        start = list(range(q.shape[0] + 1)) if row_start is None else row_start.tolist()
        u = ref.half_step(q.dtype)
        for b, s in enumerate(slots.tolist()):
            L, r = int(self.lens[s]), slice(start[b], start[b + 1])
            pos = torch.arange(L - (r.stop - r.start), L, device=q.device)
            want, tol = ref.turned(q[r], pos, rotary.frequencies, rotary.gain, rotary.rot, rotary.layout)
            within(got[r], want, tol + u * want.abs(), "q")
            want, tol = ref.turned(k[r], pos, rotary.frequencies, rotary.gain, rotary.rot, rotary.layout)
            pg, j = self.table[s].long()[pos // 16], pos % 16
            within(self.k[layer, pg, :, j], want, tol + u * want.abs(), "k")
            assert torch.equal(self.v[layer, pg, :, j], v[r])
        Checked.calls += 1
        return got


def test_every_call_of_a_session(serve, monkeypatch):
    calls = {"norm": 0, "linear": 0, "logprobs": 0}
    norm, logprobs, call = serve.rms_norm, serve.token_logprobs, LinearAttention._call

    def checked_norm(x, w, residual=None):
        want_r, y, tol = ref.norm(x, w, residual, 1e-6, 0.0, torch.bfloat16)
        got = norm(x, w, residual=residual)
        assert residual is None or torch.equal(residual, want_r)
        within(got, y, tol, "norm")
        calls["norm"] += 1
        return got

    def checked_logprobs(z, tokens, top):
        want, tol = ref.logprobs(z, tokens, top, 1.0)
        got = logprobs(z, tokens, top=top)
        for n in want:
            if n in ("rank", "top_ids"):
                assert torch.equal(got[n], want[n])
            else:
                within(got[n], want[n], tol[n], n)
        calls["logprobs"] += 1
        return got

    def checked_linear(self, fn, q, k, v, g, slots, row_start, scale, out, stream):
        before = self.state.clone()
        o = call(self, fn, q, k, v, g, slots, row_start, scale, out, stream)
        start = list(range(q.shape[0] + 1)) if row_start is None else row_start.tolist()
        spans = [(s, a, b - a) for s, a, b in zip(slots.tolist(), start, start[1:])]
        wo, to, ws, ts = ref.linear(q, k, v, g, before, spans, self.Dk ** -0.5, row_start is not None)
        within(o, wo, to, "linear attention")
        within(self.state, ws, ts, "state")
        calls["linear"] += 1
        return o

    monkeypatch.setattr(serve, "rms_norm", checked_norm)
    monkeypatch.setattr(serve, "token_logprobs", checked_logprobs)
    monkeypatch.setattr(LinearAttention, "_call", checked_linear)
    Checked.calls = 0
    tokens, _, scores, model = run(serve, cls=Checked)
    passes = 1 + 6
    assert calls == {"norm": 9 * passes, "linear": 2 * passes, "logprobs": passes} and Checked.calls == 2 * passes
    # the branches start with their two best tokens and take the best one after (torch's
    # order among equal logits is its own)
    assert torch.equal(scores[0]["rank"].view(4, 2).sort(1)[0], torch.tensor([[0, 1]] * 4, dtype=torch.int32, device="cuda"))
    assert all(torch.equal(x["logprob"], x["top_logprobs"][:, 0]) for x in scores[1:])
    assert all((s[:4] == 0).all() and (s[4:].abs().sum((1, 2, 3)) > 0).all() for s in model.states())


def test_compaction_changes_no_result(serve):
    a, b = run(serve, compact=False), run(serve, compact=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_example_command(serve, capsys, monkeypatch):
    monkeypatch.setattr("sys.argv", ["serve.py", "--steps", "4", "--branches", "2", "--hybrid"])
    serve.main()
    out = capsys.readouterr().out
    assert "3 prompts, 6 branches, 4 steps" in out and out.count("log probability -") == 6

"""Serving with the paged cache: prompts, branches and decode steps of a small
decoder whose layers are attention over a `PagedKV` and a routed-expert FFN
(`MoeLayer`). Random weights; the projections around them are plain matrix
products.

    python examples/serve.py [--steps N] [--branches N]

Three prompts of different lengths go through the layers as one chunk. Each is
forked into branches, which share the prompt's full pages and differ from their
first token on; the prompts' own slots are freed. The branches then decode
token by token, with a compaction of the pool half way. Nothing between the
prompts and the end waits for the GPU: the pages that a step needs are found
there.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from routed_expert_ffn_router_gb300 import build, synth  # noqa: E402
from routed_expert_ffn_router_gb300.layer import MoeLayer  # noqa: E402
from routed_expert_ffn_router_gb300.paged import PagedKV  # noqa: E402

BF16 = torch.bfloat16


def norm(x):
    f = x.float()
    return (f * torch.rsqrt(f.square().mean(-1, keepdim=True) + 1e-6)).to(x.dtype)


class Decoder:
    """n_layers of (attention, routed-expert FFN) around a residual stream of H."""

    def __init__(self, n_layers=4, H=512, Hq=8, Hkv=2, D=128, vocab=512, window=0, sinks=0, T_max=512, seed=0,
                 device="cuda"):
        self.n_layers, self.Hq, self.Hkv, self.D, self.window, self.sinks = n_layers, Hq, Hkv, D, window, sinks
        self.T_max, self.device = T_max, device
        g = torch.Generator().manual_seed(seed)

        def weight(*shape):
            return (torch.randn(*shape, generator=g) * shape[-2] ** -0.5).to(BF16).to(device)

        cfg = synth.MoeConfig("serve", H=H, I=256, E=32, k=4, T=16, shared_I=256, zipf_s=1.0)
        self.embed = torch.randn(vocab, H, generator=g).to(BF16).to(device)
        self.head = weight(H, vocab)
        self.wqkv = [weight(H, (Hq + 2 * Hkv) * D) for _ in range(n_layers)]
        self.wo = [weight(Hq * D, H) for _ in range(n_layers)]
        self.router = [weight(H, cfg.E) for _ in range(n_layers)]
        self.ffn = [MoeLayer(synth.make_layer(cfg, seed=seed, layer=l).to(device), T_max=T_max) for l in range(n_layers)]

    def cache(self, n_pages, page_size, n_slots, max_tokens, cls=PagedKV):
        return cls(self.n_layers, n_pages, page_size, self.Hkv, self.D, n_slots, -(-max_tokens // page_size), Hq=self.Hq,
                   max_rows=self.T_max, device=self.device)

    def __call__(self, kv, tokens, slots, row_start=None):
        """Logits of every row; tokens are the newest of their slots, whose pages
        are there (row_start None: a decode step of one token per slot)."""
        Hq, Hkv, D = self.Hq, self.Hkv, self.D
        x = self.embed[tokens]
        mask = dict(window=self.window, sinks=self.sinks)
        for l in range(self.n_layers):
            qkv = (norm(x) @ self.wqkv[l]).unflatten(1, (Hq + 2 * Hkv, D))
            q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]  # parts of one product, used in place
            kv.append(l, k, v, slots=slots, row_start=row_start)
            if row_start is None:
                o = kv.decode(l, q, slots=slots, **mask)
            else:
                o = kv.chunk(l, q, slots=slots, row_start=row_start, **mask)
            x = x + o.flatten(1) @ self.wo[l]
            h = norm(x)
            y = self.ffn[l].forward((h @ self.router[l]).float(), h)["y"]
            x = x + y.to(BF16)
        return (norm(x) @ self.head).float()

    def status(self):
        return [f.status() for f in self.ffn]


class Session:
    """Sequences of one decoder in the slots of one cache."""

    def __init__(self, model, kv):
        self.model, self.kv = model, kv

    def ints(self, values):
        return torch.tensor(values, dtype=torch.int32, device=self.model.device)

    def prompts(self, slots, prompts):
        """The prompts (lists of tokens) as one chunk; -> logits of each one's last row."""
        lens = [len(p) for p in prompts]
        start = [0]
        for n in lens:
            start.append(start[-1] + n)
        slots = self.ints(slots)
        self.kv.grow(slots, self.ints(lens))
        logits = self.model(self.kv, self.ints([t for p in prompts for t in p]), slots, self.ints(start))
        return logits[[s - 1 for s in start[1:]]]

    def fork(self, src, dst):
        self.kv.fork(self.ints(src), self.ints(dst))

    def free(self, slots):
        self.kv.free_slots(self.ints(slots))

    def step(self, slots, tokens, ones):
        """One token per slot (device tensors); -> logits."""
        self.kv.grow(slots, ones)
        return self.model(self.kv, tokens, slots)


def serve(model, kv, prompts, branches, steps, compact=True):
    """-> (tokens [steps + 1][branches of all prompts], last logits)."""
    s = Session(model, kv)
    n = len(prompts)
    logits = s.prompts(list(range(n)), prompts)
    slots = list(range(n, n + n * branches))
    s.fork([i // branches for i in range(n * branches)], slots)
    s.free(list(range(n)))
    # branch j of a prompt starts with its j-th best token
    tokens = logits.topk(branches, dim=1).indices.flatten().to(torch.int32)
    slots, ones, out = s.ints(slots), s.ints([1] * (n * branches)), [tokens]
    for i in range(steps):
        if compact and i == steps // 2:
            kv.compact()
        logits = s.step(slots, tokens, ones)
        tokens = logits.argmax(1).to(torch.int32)
        out.append(tokens)
    return torch.stack(out), logits


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=32)
    ap.add_argument("--branches", type=int, default=4)
    a = ap.parse_args()
    build.build()
    g = torch.Generator().manual_seed(1)
    prompts = [torch.randint(0, 512, (n,), generator=g).tolist() for n in (200, 41, 97)]
    model = Decoder()
    for run in range(2):  # the second is the timed one
        kv = model.cache(n_pages=512, page_size=16, n_slots=3 + 3 * a.branches, max_tokens=256 + a.steps)
        t0, t1 = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        t0.record()
        tokens, _ = serve(model, kv, prompts, a.branches, a.steps)
        t1.record()
        torch.cuda.synchronize()
        if kv.status()[0] != 0 or any(c != 0 for c, _ in model.status()):
            raise SystemExit(f"device status: {kv.status()} {model.status()}")
    print(f"{len(prompts)} prompts, {tokens.shape[1]} branches, {a.steps} steps: {t0.elapsed_time(t1):.1f} ms, "
          f"{kv.table.shape[1]} pages per slot, {512 - int(kv.n_free)} pages in use")
    for j in range(tokens.shape[1]):
        print(f"prompt {j // a.branches} branch {j % a.branches}:", " ".join(map(str, tokens[:12, j].tolist())), "...")


if __name__ == "__main__":
    main()

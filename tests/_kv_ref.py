"""Plain 64-bit reference of the paged cache's attention and page operations,
and the builder of poisoned test caches (test infrastructure only)."""
import math

import torch

GARBAGE = (-1, -7, 1 << 30, 2147483647)


class Case:
    """A cache of one or two layers holding B sequences in shuffled pages, and
    the rows of one call. Everything that no row may use is NaN or a garbage
    page number: unused pages, the rest of last pages, tokens outside every
    row's window, table entries past the length."""

    def __init__(self, lens, news, Hq, Hkv, D, page, dtype=torch.bfloat16, window=0, sinks=0, n_layers=1, seed=0,
                 dev="cuda", poison=True, q_gain=1.5, v_mean=0.0, spare_pages=3):
        g = torch.Generator().manual_seed(seed + 1)
        self.lens_l, self.news_l = list(lens), list(news)
        self.Hq, self.Hkv, self.D, self.page, self.dtype = Hq, Hkv, D, page, dtype
        self.window, self.sinks, self.dev = window, sinks, dev
        B = len(lens)
        used = [-(-n // page) for n in lens]
        self.n_pages = sum(used) + spare_pages
        self.max_pages = max(used + [1]) + 2
        self.n_slots = B + 2
        fill = float("nan") if poison else 0.0
        shape = (n_layers, self.n_pages, Hkv, page, D)
        k = torch.full(shape, fill, dtype=dtype)
        v = torch.full(shape, fill, dtype=dtype)
        table = torch.tensor(GARBAGE, dtype=torch.int32)[torch.randint(0, 4, (self.n_slots, self.max_pages), generator=g)]
        order = torch.randperm(self.n_pages, generator=g)
        self.slots = torch.randperm(self.n_slots, generator=g)[:B].to(torch.int32)
        lens_t = torch.zeros(self.n_slots, dtype=torch.int32)
        refs = torch.zeros(self.n_pages, dtype=torch.int32)
        at = 0
        for b in range(B):
            s, L, n = int(self.slots[b]), lens[b], news[b]
            lens_t[s] = L
            pg = order[at:at + used[b]]
            at += used[b]
            refs[pg] = 1
            see = self.seen(L, n)
            for i in range(used[b]):
                rows = see[i * page:(i + 1) * page]
                if rows.any():
                    table[s, i] = pg[i]
                    r = rows.nonzero()[:, 0]
                    for pool in (k, v):
                        x = torch.randn(n_layers, Hkv, len(r), D, generator=g)
                        if pool is v:
                            x += v_mean
                        pool[:, pg[i].item()][:, :, r] = x.to(dtype)
        self.free = torch.zeros(self.n_pages, dtype=torch.int32)
        self.free[:self.n_pages - at] = order[at:].to(torch.int32)
        self.n_free = torch.tensor([self.n_pages - at], dtype=torch.int32)
        self.k, self.v, self.table, self.lens, self.refs = k, v, table, lens_t, refs
        T = sum(news)
        self.T = T
        # q is a part of a wider projection: row stride (Hq + 3) * D
        self.q_wide = (torch.randn(T, Hq + 3, D, generator=g) * q_gain).to(dtype)
        self.row_start = torch.tensor([0] + list(torch.tensor(news).cumsum(0)), dtype=torch.int32)
        self.to(dev)

    def to(self, dev):
        for n in ("k", "v", "table", "lens", "refs", "free", "n_free", "q_wide", "row_start", "slots"):
            setattr(self, n, getattr(self, n).to(dev))
        self.q = self.q_wide[:, 1:1 + self.Hq]

    def seen(self, L, n):
        """bool [pages * page]: tokens that some row of a sequence sees."""
        see = torch.zeros(-(-L // self.page) * self.page, dtype=torch.bool)
        for p in range(max(0, L - n), L):
            if not self.window:
                see[:p + 1] = True
            else:
                see[max(0, p - self.window + 1):p + 1] = True
                see[:min(self.sinks, p + 1)] = True
        return see

    def cache(self, max_rows=None):
        from routed_expert_ffn_router_gb300.paged import PagedKV
        return PagedKV.over(self.k, self.v, self.table, self.lens, self.refs, self.free, self.n_free, Hq=self.Hq,
                            max_rows=self.T if max_rows is None else max_rows)

    def reference(self, layer=0, scale=None):
        """-> o, lse, tol_o, tol_lse in float64. The tolerances: u = half a step of the type.
        Output rounding u |o|; probabilities rounded to the type, u A with A = sum p |v|;
        scores from D fp32 products (2^-23 each, the tensor cores' sums may truncate), an
        error d in a score changing p by up to 2 d; fp32 sums of n terms."""
        scale = self.D ** -0.5 if scale is None else scale
        u = torch.finfo(self.dtype).eps / 2
        dev, G = self.k.device, self.Hq // self.Hkv
        o = torch.zeros(self.T, self.Hq, self.D, dtype=torch.float64, device=dev)
        lse = torch.full((self.T, self.Hq), -math.inf, dtype=torch.float64, device=dev)
        tol_o, tol_l = torch.zeros_like(o), torch.zeros_like(lse)
        start = self.row_start.tolist()
        for b, s in enumerate(self.slots.tolist()):
            L, n = self.lens_l[b], self.news_l[b]
            if L == 0 or n == 0:
                continue
            see = self.seen(L, n)[:L].to(dev)
            tok = see.nonzero()[:, 0]
            pg = self.table[s].long()[tok // self.page]
            pos = torch.arange(L - n, L, device=dev)
            hide = tok[None] > pos[:, None]
            if self.window:
                hide |= (tok[None] <= pos[:, None] - self.window) & (tok[None] >= self.sinks)
            for h in range(self.Hkv):
                kh = self.k[layer, pg, h, tok % self.page].double()
                vh = self.v[layer, pg, h, tok % self.page].double()
                for a in range(G):
                    qh = self.q[start[b]:start[b + 1], h * G + a].double()
                    x = (qh @ kh.T) * scale
                    x[hide] = -math.inf
                    z = torch.logsumexp(x, 1)
                    p = torch.exp(x - torch.where(z == -math.inf, torch.zeros_like(z), z)[:, None])
                    vis = p @ torch.nan_to_num(vh, nan=0.0, posinf=0.0, neginf=0.0)
                    bad = ~torch.isfinite(vh)
                    if bad.any():  # a non-finite value reaches the rows that see it, and no others
                        w = torch.where(hide[:, :, None], torch.zeros((), dtype=torch.float64, device=dev), p[:, :, None] * vh[None])
                        vis = w.sum(1)
                    o[start[b]:start[b + 1], h * G + a] = vis
                    lse[start[b]:start[b + 1], h * G + a] = z
                    amp = (qh.abs() @ kh.abs().T).amax(1) * abs(scale)  # of one score
                    d = (self.D + 16) * 2.0 ** -23 * amp + 2.0 ** -20
                    A = p @ torch.nan_to_num(vh, nan=0.0, posinf=0.0, neginf=0.0).abs()
                    few = (len(tok) + 64) * 2.0 ** -23
                    tol_o[start[b]:start[b + 1], h * G + a] = 1.05 * (u * vis.abs() + (u + 2 * d + few)[:, None] * A) + 1e-30
                    tol_l[start[b]:start[b + 1], h * G + a] = d + few + 2.0 ** -22 * z.abs()
        return o, lse, tol_o, tol_l


def check(case, got, want, what=""):
    o, lse = got
    ro, rl, to, tl = want
    # an fp16 result below the normal range has a fixed step
    tiny = torch.finfo(case.dtype).smallest_normal * torch.finfo(case.dtype).eps
    empty = torch.isinf(rl)
    assert torch.equal(torch.isneginf(lse.double()), empty), what + ": rows that see nothing"
    assert (o[empty] == 0).all(), what + ": rows that see nothing give zeros"
    fin = torch.isfinite(ro)
    assert torch.equal(torch.isfinite(o), fin), what + ": finite where the definition is"
    err = ((o.double() - ro).abs() - to - tiny)[fin]
    assert err.numel() == 0 or err.max() <= 0, f"{what}: o beyond its bound by {err.max():.3e}"
    el = ((lse.double() - rl).abs() - tl)[~empty]
    assert el.numel() == 0 or el.max() <= 0, f"{what}: lse beyond its bound by {el.max():.3e}"


# ------------------------------------------------------------------ page operations on host lists
class Books:
    """The page operations, step by step on Python lists and CPU tensors."""

    def __init__(self, k, v, table, lens, refs, free, n_free):
        self.k, self.v = k.cpu().clone(), v.cpu().clone()
        self.page = k.shape[3]
        self.table, self.lens, self.refs = table.tolist(), lens.tolist(), refs.tolist()
        self.rest = free.tolist()
        self.stack = self.rest[:int(n_free)]

    def n(self, length):
        return -(-length // self.page)

    def pop(self):
        return self.stack.pop()

    def push(self, p):
        self.stack.append(p)
        self.rest[len(self.stack) - 1] = p

    def grow(self, slots, add):
        for s, a in zip(slots, add):
            for c in range(self.n(self.lens[s]), self.n(self.lens[s] + a)):
                self.table[s][c] = self.pop()
                self.refs[self.table[s][c]] = 1
            self.lens[s] += a

    def fork(self, src, dst):
        for a, b in zip(src, dst):
            full, rows = divmod(self.lens[a], self.page)
            for c in range(full):
                self.table[b][c] = self.table[a][c]
                self.refs[self.table[a][c]] += 1
            if rows:
                p, q = self.pop(), self.table[a][full]
                self.refs[p], self.table[b][full] = 1, p
                self.k[:, p, :, :rows] = self.k[:, q, :, :rows]
                self.v[:, p, :, :rows] = self.v[:, q, :, :rows]
            self.lens[b] = self.lens[a]

    def free(self, slots):
        gone = []
        for s in slots:
            for c in range(self.n(self.lens[s])):
                p = self.table[s][c]
                self.refs[p] -= 1
                if self.refs[p] == 0:
                    gone.append(p)
            self.lens[s], self.table[s] = 0, [-1] * len(self.table[s])
        for p in sorted(gone, reverse=True):
            self.push(p)

    def compact(self):
        live = [p for p, r in enumerate(self.refs) if r > 0]
        n = len(live)
        moves = dict(zip([p for p in live if p >= n], [p for p in range(n) if self.refs[p] == 0]))
        for a, b in moves.items():
            self.k[:, b], self.v[:, b] = self.k[:, a], self.v[:, a]
            self.refs[b], self.refs[a] = self.refs[a], 0
        for s, length in enumerate(self.lens):
            for c in range(self.n(length)):
                self.table[s][c] = moves.get(self.table[s][c], self.table[s][c])
        self.stack = list(range(len(self.refs) - 1, n - 1, -1))
        self.rest[:len(self.stack)] = self.stack
        return len(moves)

    def copy(self, src, dst):
        self.k[:, dst], self.v[:, dst] = self.k[:, src], self.v[:, src]

    def check(self, kv, what=""):
        assert int(kv.n_free) == len(self.stack), what + ": free pages"
        assert kv.lens.tolist() == self.lens, what + ": lens"
        assert kv.refs.tolist() == self.refs, what + ": refs"
        assert kv.free.tolist() == self.rest, what + ": the free stack"
        assert kv.table.tolist() == self.table, what + ": tables"
        for a, b, n in ((kv.k, self.k, "k"), (kv.v, self.v, "v")):
            assert torch.equal(a.cpu().view(torch.int16), b.view(torch.int16)), what + ": pool " + n

"""The paged key-value cache and its attention, as cases that can be timed and checked.

Three operators, each in a plain torch form (`own` false) and as the calls that a
program makes of this package (`own` true):

  decode  the new tokens' K/V rows are written into their pages, then each row of
          a decode window attends over its sequence's pages (optionally a sliding
          window plus a few first tokens that stay visible);
  chunk   the same for prompt chunks: many new tokens per sequence, causal;
  pages   "fork": sequences are forked (full pages shared, the last page's rows
          copied) and the forks freed; "compact": a group of sequences is freed,
          the live pages move to the low page ids and the group is admitted again.

Cache layout: k, v [layers][pages][kv heads][page][D]; table int32 [slots][max
pages] (-1 = none), lens int32 [slots] (new tokens included), refs int32 [pages],
a stack of free pages. Sequence lengths are a function of the case alone; pages,
values and the order of pages come from the seed.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------ cases
def _decode(name, B, max_len, Hq, Hkv, D=128, page=16, n_q=1, dtype="bf16", window=0, sinks=0, ragged=True):
    return dict(name=name, op="decode", B=B, max_len=max_len, Hq=Hq, Hkv=Hkv, D=D, page=page, n_q=n_q,
                dtype=dtype, window=window, sinks=sinks, ragged=ragged)


def _chunk(name, B, new, max_len, Hq, Hkv, D=128, page=16, dtype="bf16", window=0, sinks=0, ragged=True):
    return dict(name=name, op="chunk", B=B, new=new, max_len=max_len, Hq=Hq, Hkv=Hkv, D=D, page=page,
                dtype=dtype, window=window, sinks=sinks, ragged=ragged)


def _pages(name, what, layers, B, max_len, Hkv, D=128, page=16, n=4, dtype="bf16"):
    return dict(name=name, op="pages", what=what, layers=layers, B=B, max_len=max_len, Hkv=Hkv, D=D,
                page=page, n=n, dtype=dtype)


def listed():
    return [
        # one conversation's next token over a short context: the call's latency
        _decode("decode_one", 1, 517, 16, 4),
        # a decode window of 8 conversations of different lengths
        _decode("decode_window", 8, 4093, 16, 2),
        # 16 rows, token + proposal for 8 conversations, with a sliding window and 4 first tokens
        _decode("decode_pairs_sliding", 8, 16001, 32, 8, page=32, n_q=2, dtype="fp16", window=1024, sinks=4),
        # one conversation with a very long context: the length is what can be split
        _decode("decode_long", 1, 131057, 32, 8, page=64, ragged=False),
        # a full server: 64 conversations of different lengths
        _decode("decode_batch", 64, 8191, 32, 8),
        # a short question: 40 tokens without context
        _chunk("chunk_short", 1, 40, 40, 16, 4, D=64, dtype="fp16", ragged=False),
        # a prompt chunk of 2,048 tokens at the start of its sequence
        _chunk("chunk_prompt", 1, 2048, 2048, 16, 4, ragged=False),
        # several prompts of different lengths at once, sliding window and 4 first tokens
        _chunk("chunk_ragged_sliding", 5, 901, 6011, 28, 4, page=32, window=512, sinks=4),
        # a later chunk of a long document: 2,048 tokens over 32,741 of context
        _chunk("chunk_long", 1, 2048, 32741, 32, 8, page=64, ragged=False),
        # a conversation forked into 4 branches, over the 48 layers of a stack
        _pages("fork_branches", "fork", 48, 2, 1003, 2, n=4),
        # 64 forks at once (best-of-n sampling on a batch)
        _pages("fork_batch", "fork", 48, 16, 1511, 4, page=32, n=64),
        # finished sequences leave, the others' pages are packed together, new ones are admitted
        _pages("compact_pool", "compact", 48, 24, 1777, 4, page=32, n=12),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["decode", "decode", "chunk", "chunk", "pages"])
    Hq, Hkv = rng.choice([(16, 4), (16, 2), (32, 8), (8, 8), (28, 4), (12, 4), (32, 2), (24, 1), (5, 5)])
    D = rng.choice([64, 128, 128])
    page = rng.choice([16, 32, 64])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    window, sinks = rng.choice([(0, 0), (0, 0), (_logint(rng, 16, 4096), rng.choice([0, 1, 4, 37]))])
    if op == "decode":
        B = _logint(rng, 1, 64)
        n_q = rng.choice([1, 1, 1, 2, 3])
        most = max(2, min(65536, int(64 * 8191 * 8 * 128 * 0.5 / (B * Hkv * D))))
        c = _decode("", B, _logint(rng, 1, most), Hq, Hkv, D, page, n_q, dtype, window, sinks, rng.random() < 0.7)
    elif op == "chunk":
        B = rng.choice([1, 1, 2, 3, 7])
        new = _logint(rng, 2, 2048)
        most = max(new + 1, min(32741, int(2048 * 32741 * 32 * 0.8 / (B * new * Hq))))
        c = _chunk("", B, new, _logint(rng, new, most), Hq, Hkv, D, page, dtype, window, sinks, rng.random() < 0.6)
    else:
        what = rng.choice(["fork", "compact"])
        layers = rng.choice([1, 4, 24, 48])
        B = rng.randint(2, 16)
        n = rng.randint(1, 48) if what == "fork" else max(1, B // 2)
        c = _pages("", what, layers, B, _logint(rng, 3, 1511), rng.choice([1, 2, 4]), D, page, n, dtype)
    c.pop("name")
    return c


def _spread(n, lo, hi):
    """n lengths over [lo, hi], the longest first, from a fixed low-discrepancy sequence."""
    return [hi if i == 0 else max(lo, int(lo + (hi - lo) * ((i * 0.6180339887498949) % 1.0))) for i in range(n)]


def _lens(case):
    """The sequences' lengths, new tokens included."""
    if case["op"] == "decode":
        L = _spread(case["B"], case["max_len"] // 8, case["max_len"]) if case["ragged"] else [case["max_len"]] * case["B"]
        return [max(case["n_q"], x) for x in L]
    if case["op"] == "chunk":
        return [max(n, m) for n, m in zip(_news(case), _spread(case["B"], case["max_len"] // 3, case["max_len"]))] \
            if case["ragged"] else [max(case["new"], case["max_len"])] * case["B"]
    return _spread(case["B"], max(1, case["max_len"] // 4), case["max_len"])


def _news(case):
    """New tokens per sequence."""
    if case["op"] == "decode":
        return [case["n_q"]] * case["B"]
    return _spread(case["B"], max(1, case["new"] // 5), case["new"]) if case["ragged"] else [case["new"]] * case["B"]


def _visible_pairs(n, L, W, S):
    """(query, key) pairs of n queries at the end of L keys, and the keys any of them sees."""
    pairs, first = 0, max(0, L - n)
    for p in range(first, L):
        if not W or p + 1 <= W:
            pairs += p + 1
        else:
            lo = p - W + 1
            pairs += W + min(S, lo)
    lo = max(0, first - W + 1) if W else 0
    return pairs, L - lo + min(S, lo)


def work(case):
    el = 2
    if case["op"] == "pages":
        page_row = case["layers"] * 2 * case["Hkv"] * case["D"] * el
        L = _lens(case)
        if case["what"] == "fork":
            rows = sum(L[i % case["B"]] % case["page"] for i in range(case["n"]))
            return {"bytes": 2 * rows * page_row + 4 * (sum(L) // case["page"] + case["n"]), "flops": 0}
        n_pg = [-(-x // case["page"]) for x in L]
        moved = min(sum(n_pg[:case["n"]]), sum(n_pg[case["n"]:]))
        return {"bytes": 2 * moved * case["page"] * page_row, "flops": 0}
    flops = nbytes = 0
    for n, L in zip(_news(case), _lens(case)):
        pairs, keys = _visible_pairs(n, L, case["window"], case["sinks"])
        flops += 4 * pairs * case["Hq"] * case["D"]
        nbytes += 2 * keys * case["Hkv"] * case["D"] * el                       # K and V that are seen
        nbytes += 2 * min(n, L) * (case["Hq"] + case["Hkv"]) * case["D"] * el   # q, o; new K, V into their pages
    return {"bytes": nbytes, "flops": flops}


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed) * 7919 + 11)
    dt, page, D, Hkv = DTYPES[case["dtype"]], case["page"], case["D"], case["Hkv"]
    L, layers = _lens(case), case.get("layers", 1)
    used = [-(-x // page) for x in L]
    more = 3 if case["op"] != "pages" else case["n"] + 8 if case["what"] == "fork" else sum(used) // 4 + 1
    n_pages = sum(used) + more
    slots = case["B"] + (case["n"] if case["op"] == "pages" else 1)
    max_pages = max(used) + 2

    def randn(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32) * std).to(dt)

    k = torch.empty(layers, n_pages, Hkv, page, D, dtype=dt, device=DEV)
    v = torch.empty_like(k)
    for i in range(layers):
        k[i], v[i] = randn(n_pages, Hkv, page, D), randn(n_pages, Hkv, page, D)
    order = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    table = torch.full((slots, max_pages), -1, dtype=torch.int32, device=DEV)
    refs = torch.zeros(n_pages, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(used):
        table[b, :n] = order[at:at + n]
        at += n
    refs[order[:at].long()] = 1
    lens = torch.zeros(slots, dtype=torch.int32, device=DEV)
    lens[:len(L)] = torch.tensor(L, dtype=torch.int32, device=DEV)
    free = torch.zeros(n_pages, dtype=torch.int32, device=DEV)
    free[:n_pages - at] = order[at:]
    n_free = torch.full((1,), n_pages - at, dtype=torch.int32, device=DEV)
    s = dict(case=case, k=k, v=v, table=table, lens=lens, refs=refs, free=free, n_free=n_free, passes=0)
    if case["op"] == "pages":
        if case["what"] == "fork":
            s["src"] = (torch.arange(case["n"], device=DEV) % case["B"]).to(torch.int32)
            s["dst"] = (torch.arange(case["n"], device=DEV) + case["B"]).to(torch.int32)
        else:  # the two groups take turns: the one admitted longest ago leaves
            ids = torch.arange(case["B"], device=DEV, dtype=torch.int32)
            s["groups"] = [ids[:case["n"]].contiguous(), ids[case["n"]:].contiguous()]
            s["adds"] = [lens[i.long()].clone() for i in s["groups"]]
        return s
    new = _news(case)
    T = sum(new)
    # q, k and v of the new tokens are parts of one projection's output, as a model makes them
    qkv = randn(T, case["Hq"] + 2 * Hkv, D)
    s["q"] = qkv[:, :case["Hq"]]
    s["q"] *= 1.5
    s["k_new"] = qkv[:, case["Hq"]:case["Hq"] + Hkv]
    s["v_new"] = qkv[:, case["Hq"] + Hkv:]
    s["slots"] = torch.randperm(case["B"], generator=g, device=DEV).to(torch.int32)
    # the i-th group of rows belongs to slot slots[i]; lengths and new tokens go by the slot
    new = torch.tensor(new, dtype=torch.int32, device=DEV)[s["slots"].long()]
    s["row_start"] = torch.cat([new.new_zeros(1), new.cumsum(0).to(torch.int32)])
    s["scale"] = D ** -0.5
    return s


# ------------------------------------------------------------------ the plain forms
def _rows(s):
    """For the padded form: row index [B][Tm] of each query, whether there is one, its position; and each row's (b, i)."""
    case = s["case"]
    start = s["row_start"].long()
    n = start[1:] - start[:-1]
    i = torch.arange(max(_news(case)), device=DEV)
    t = torch.arange(s["q"].shape[0], device=DEV)
    b_of = (t[:, None] >= start[None, 1:]).sum(1)
    pos = s["lens"][s["slots"].long()].long()[:, None] - n[:, None] + i[None]
    return (start[:-1, None] + i[None]).clamp(max=t.numel() - 1), i[None] < n[:, None], pos, b_of, t - start[b_of]


def _plain_attention(s):
    case = s["case"]
    page, Hkv, D, W = case["page"], case["Hkv"], case["D"], case["window"]
    G = case["Hq"] // Hkv
    k, v, slots = s["k"][0], s["v"][0], s["slots"].long()
    idx, real, pos, b_of, i_of = _rows(s)
    # the new rows into their pages
    p = pos[b_of, i_of]
    pg = s["table"][slots[b_of], p // page].long()
    k[pg, :, p % page] = s["k_new"]
    v[pg, :, p % page] = s["v_new"]
    # every sequence's keys and values, padded to the longest
    n_pg = -(-max(_lens(case)) // page)
    tab = s["table"][slots, :n_pg].long().clamp(min=0)
    kk = k[tab].permute(0, 2, 1, 3, 4).reshape(len(slots), Hkv, n_pg * page, D).float()
    vv = v[tab].permute(0, 2, 1, 3, 4).reshape(len(slots), Hkv, n_pg * page, D).float()
    q = s["q"][idx].float()                                        # [B][Tm][Hq][D]
    Tm = q.shape[1]
    q = q.reshape(len(slots), Tm, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(len(slots), Hkv, G * Tm, D)
    x = torch.matmul(q, kk.transpose(2, 3)) * s["scale"]           # [B][Hkv][G Tm][L]
    j = torch.arange(n_pg * page, device=DEV)
    see = real[:, :, None] & (j <= pos[:, :, None])
    if W:
        see &= (j > pos[:, :, None] - W) | (j < case["sinks"])
    x = x.reshape(len(slots), Hkv, G, Tm, -1)
    x = x.masked_fill_(~see[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    e = x.sub_(m).exp_()
    l = e.sum(-1, keepdim=True)
    lse = torch.log(l) + m
    e = e.reshape(len(slots), Hkv, G * Tm, -1)
    vv = vv.masked_fill((j >= s["lens"][slots][:, None])[:, None, :, None], 0.0)
    o = torch.matmul(e, vv).reshape(len(slots), Hkv, G, Tm, D) / torch.where(l == 0, torch.ones_like(l), l)
    o = o.permute(0, 3, 1, 2, 4).reshape(len(slots), Tm, case["Hq"], D)[b_of, i_of].to(k.dtype)
    lse = lse[..., 0].permute(0, 3, 1, 2).reshape(len(slots), Tm, case["Hq"])[b_of, i_of]
    return {"o": o, "lse": lse, "k": s["k"], "v": s["v"]}


def _cols(s):
    return torch.arange(s["table"].shape[1], device=DEV)


def _plain_fork(s, src, dst):
    page, table, refs = s["case"]["page"], s["table"], s["refs"]
    L = s["lens"][src.long()].long()
    full, rest = L // page, L % page
    need = rest > 0
    rank = need.long().cumsum(0) - 1
    rows = table[src.long()].long()
    last = rows.gather(1, full.clamp(max=rows.shape[1] - 1)[:, None])[:, 0].clamp(min=0)
    new = torch.where(need, s["free"][(s["n_free"].long() - 1 - rank).clamp(min=0)].long(), last)
    shared = _cols(s)[None] < full[:, None]
    tail = (_cols(s)[None] == full[:, None]) & need[:, None]
    table[dst.long()] = torch.where(shared, rows, torch.where(tail, new[:, None], torch.full_like(rows, -1))).int()
    refs.index_add_(0, torch.where(shared, rows, 0).flatten(), shared.flatten().int())
    refs.index_add_(0, torch.where(need, new, 0), need.int())
    s["lens"][dst.long()] = L.int()
    s["n_free"] -= need.sum().int()
    take = (torch.arange(page, device=DEV)[None] < rest[:, None])[None, :, None, :, None]
    for pool in (s["k"], s["v"]):
        pool[:, new] = torch.where(take, pool[:, last], pool[:, new])


def _plain_free(s, slots):
    page, refs, free = s["case"]["page"], s["refs"], s["free"]
    rows = s["table"][slots.long()].long()
    held = _cols(s)[None] < -(-s["lens"][slots.long()].long() // page)[:, None]
    before = refs.clone()
    refs.index_add_(0, torch.where(held, rows, 0).flatten(), -held.flatten().int())
    gone = (before > 0) & (refs == 0)
    rank, n = gone.long().cumsum(0) - 1, gone.sum()
    at = torch.where(gone, s["n_free"].long() + n - 1 - rank, refs.numel())
    longer = torch.cat([free, free.new_zeros(1)])
    longer[at] = torch.arange(refs.numel(), device=DEV, dtype=torch.int32)
    free.copy_(longer[:-1])
    s["n_free"] += n.int()
    s["lens"][slots.long()] = 0
    s["table"][slots.long()] = -1


def _plain_grow(s, slots, add):
    page = s["case"]["page"]
    L = s["lens"][slots.long()].long()
    a, b = -(-L // page), -(-(L + add.long()) // page)
    first = (b - a).cumsum(0) - (b - a)
    fresh = (_cols(s)[None] >= a[:, None]) & (_cols(s)[None] < b[:, None])
    rank = first[:, None] + _cols(s)[None] - a[:, None]
    page_id = s["free"][(s["n_free"].long() - 1 - rank).clamp(min=0)].long()
    s["table"][slots.long()] = torch.where(fresh, page_id.int(), s["table"][slots.long()])
    s["refs"].index_add_(0, torch.where(fresh, page_id, 0).flatten(), fresh.flatten().int())
    s["lens"][slots.long()] = (L + add).int()
    s["n_free"] -= (b - a).sum().int()


def _plain_compact(s):
    page, refs, table = s["case"]["page"], s["refs"], s["table"]
    ids = torch.arange(refs.numel(), device=DEV)
    live = refs > 0
    n_live = live.sum()
    to, frm = (~live & (ids < n_live)).nonzero()[:, 0], (live & (ids >= n_live)).nonzero()[:, 0]
    remap = ids.clone()
    remap[frm] = to
    for pool in (s["k"], s["v"]):
        pool[:, to] = pool[:, frm]
    held = _cols(s)[None] < -(-s["lens"].long() // page)[:, None]
    table.copy_(torch.where(held, remap[table.long().clamp(min=0)].int(), table))
    refs.copy_(torch.zeros_like(refs).index_add_(0, remap, refs))
    s["free"].copy_(torch.where(ids < refs.numel() - n_live, (refs.numel() - 1 - ids).int(), s["free"]))
    s["n_free"].copy_((refs.numel() - n_live).int()[None])


def _meta(s):
    return {n: s[n] for n in ("k", "v", "table", "lens", "refs", "free", "n_free")}


# ------------------------------------------------------------------ one pass
def _handle(s):
    """The cache object that a program keeps, over the state's buffers."""
    if "kv" not in s:
        from routed_expert_ffn_router_gb300.paged import PagedKV
        s["kv"] = PagedKV.over(s["k"], s["v"], s["table"], s["lens"], s["refs"], s["free"], s["n_free"],
                               Hq=s["case"].get("Hq", s["case"]["Hkv"]), max_rows=s["q"].shape[0] if "q" in s else 0)
    return s["kv"]


def run(s):
    case = s["case"]
    if case["op"] == "pages":
        turn, s["passes"] = s["passes"] % 2, s["passes"] + 1
        if case["what"] == "fork":
            if own:
                kv = _handle(s)
                kv.fork(s["src"], s["dst"])
                kv.free_slots(s["dst"])
            else:
                _plain_fork(s, s["src"], s["dst"])
                _plain_free(s, s["dst"])
        elif own:
            kv = _handle(s)
            kv.free_slots(s["groups"][turn])
            kv.compact()
            kv.grow(s["groups"][turn], s["adds"][turn])
        else:
            _plain_free(s, s["groups"][turn])
            _plain_compact(s)
            _plain_grow(s, s["groups"][turn], s["adds"][turn])
        return _meta(s)
    if not own:
        return _plain_attention(s)
    kv = _handle(s)
    if case["op"] == "decode":
        kv.append(0, s["k_new"], s["v_new"], slots=s["slots"])
        o, lse = kv.decode(0, s["q"], slots=s["slots"], scale=s["scale"], window=case["window"],
                           sinks=case["sinks"], want_lse=True)
    else:
        kv.append(0, s["k_new"], s["v_new"], slots=s["slots"], row_start=s["row_start"])
        o, lse = kv.chunk(0, s["q"], slots=s["slots"], row_start=s["row_start"], scale=s["scale"],
                          window=case["window"], sinks=case["sinks"], want_lse=True)
    return {"o": o, "lse": lse, "k": s["k"], "v": s["v"]}


# ------------------------------------------------------------------ the definition, in 64 bits
def _exact_pages(s):
    """The page operations step by step on host lists."""
    case, page = s["case"], s["case"]["page"]
    table, lens, refs = s["table"].tolist(), s["lens"].tolist(), s["refs"].tolist()
    stack, rest = s["free"].tolist()[:int(s["n_free"])], s["free"].tolist()
    k, v = s["k"], s["v"]

    def leave(slots):
        gone = []
        for b in slots:
            for c in range(-(-lens[b] // page)):
                p = table[b][c]
                refs[p] -= 1
                if refs[p] == 0:
                    gone.append(p)
            lens[b], table[b] = 0, [-1] * len(table[b])
        for p in sorted(gone, reverse=True):
            stack.append(p)
            rest[len(stack) - 1] = p

    if case["what"] == "fork":
        src, dst = s["src"].tolist(), s["dst"].tolist()
        for a, b in zip(src, dst):
            n, r = lens[a] // page, lens[a] % page
            for c in range(n):
                table[b][c] = table[a][c]
                refs[table[a][c]] += 1
            if r:
                p = stack.pop()
                refs[p], table[b][n] = 1, p
                k[:, p, :, :r] = k[:, table[a][n], :, :r]
                v[:, p, :, :r] = v[:, table[a][n], :, :r]
            lens[b] = lens[a]
        leave(dst)
    else:
        slots, adds = s["groups"][0].tolist(), s["adds"][0].tolist()
        leave(slots)
        alive = [p for p in range(len(refs)) if refs[p] > 0]
        holes = [p for p in range(len(alive)) if refs[p] == 0]
        moves = dict(zip([p for p in alive if p >= len(alive)], holes))
        for a, b in moves.items():
            k[:, b], v[:, b] = k[:, a], v[:, a]
            refs[b], refs[a] = refs[a], 0
        for b in range(len(lens)):
            for c in range(-(-lens[b] // page)):
                table[b][c] = moves.get(table[b][c], table[b][c])
        stack[:] = range(len(refs) - 1, len(alive) - 1, -1)
        rest[:len(stack)] = stack
        for b, n in zip(slots, adds):
            for c in range(-(-lens[b] // page), -(-(lens[b] + n) // page)):
                table[b][c] = stack.pop()
                refs[table[b][c]] = 1
            lens[b] += n
    return {"k": k.double(), "v": v.double(), "table": torch.tensor(table), "lens": torch.tensor(lens),
            "refs": torch.tensor(refs), "free": torch.tensor(rest), "n_free": torch.tensor([len(stack)])}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "pages":
        return _exact_pages(s)
    page, Hkv, W, S = case["page"], case["Hkv"], case["window"], case["sinks"]
    G = case["Hq"] // Hkv
    start, order = s["row_start"].tolist(), s["slots"].tolist()
    T = s["q"].shape[0]
    o = torch.zeros(T, case["Hq"], case["D"], dtype=torch.float64, device=DEV)
    lse = torch.full((T, case["Hq"]), -math.inf, dtype=torch.float64, device=DEV)
    k, v = s["k"][0], s["v"][0]
    for i, b in enumerate(order):
        L, n = int(s["lens"][b]), start[i + 1] - start[i]
        for p0 in range(L - n, L):  # one page's part of the new rows at a time
            if p0 % page and p0 > L - n:
                continue
            m = min(page - p0 % page, L - p0)
            at, pg = start[i] + p0 - (L - n), int(s["table"][b, p0 // page])
            k[pg, :, p0 % page:p0 % page + m] = s["k_new"][at:at + m].transpose(0, 1)
            v[pg, :, p0 % page:p0 % page + m] = s["v_new"][at:at + m].transpose(0, 1)
    for i, b in enumerate(order):
        L, n = int(s["lens"][b]), start[i + 1] - start[i]
        pages = s["table"][b, :-(-L // page)].long()
        j = torch.arange(L, device=DEV)
        pos = torch.arange(L - n, L, device=DEV)
        hide = j[None] > pos[:, None]
        if W:
            hide |= (j[None] <= pos[:, None] - W) & (j[None] >= S)
        for h in range(Hkv):
            kh = k[pages, h].reshape(-1, case["D"])[:L].double()
            vh = v[pages, h].reshape(-1, case["D"])[:L].double()
            for a in range(G):
                x = s["q"][start[i]:start[i + 1], h * G + a].double() @ kh.T * s["scale"]
                x[hide] = -math.inf
                z = torch.logsumexp(x, 1)
                lse[start[i]:start[i + 1], h * G + a] = z
                pr = torch.exp(x - torch.where(z == -math.inf, torch.zeros_like(z), z)[:, None])
                o[start[i]:start[i + 1], h * G + a] = pr @ vh
    return {"o": o, "lse": lse, "k": s["k"].double(), "v": s["v"].double()}

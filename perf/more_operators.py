"""What stands around the attention and the experts of a decoder layer, as cases that
can be timed and checked.

Four operators, each in a plain torch form (`own` false) and as the calls that a
program makes of this package (`own` true):

  norm      the residual's addition and the root-mean-square norm of the sum, in 16
            bits or in e4m3 with a scale for each row or group of columns;
  rope      rotary positions of new queries and keys, the keys and the values written
            into their pages of the cache;
  logprobs  log probabilities of given tokens, their ranks, the rows' entropies and
            the top alternatives;
  linear    linear attention with a decay for each head and token: "step" for decode
            windows, "chunk" for prompts, over a state per sequence.

Sequence lengths are a function of the case alone; values and places come from the seed.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
E4M3 = torch.float8_e4m3fn
EPS = 1e-6


# ------------------------------------------------------------------ cases
def _norm(name, T, H, x="bf16", res="bf16", out="bf16", group=0):
    return dict(name=name, op="norm", T=T, H=H, x=x, res=res, out=out, group=group)


def _rope(name, B, new, max_len, Hq, Hkv, D=128, rot=128, layout="half", scaling="none", page=16, dtype="bf16",
          ragged=True):
    return dict(name=name, op="rope", B=B, new=new, max_len=max_len, Hq=Hq, Hkv=Hkv, D=D, rot=rot, layout=layout,
                scaling=scaling, page=page, dtype=dtype, ragged=ragged)


def _logprobs(name, T, V, top, dtype="bf16", pad=0, masked=0.0, temperature=1.0):
    return dict(name=name, op="logprobs", T=T, V=V, top=top, dtype=dtype, pad=pad, masked=masked,
                temperature=temperature)


def _linear(name, what, B, new, Hk, Hv, D=128, dtype="bf16", ragged=True):
    return dict(name=name, op="linear", what=what, B=B, new=new, Hk=Hk, Hv=Hv, D=D, dtype=dtype, ragged=ragged)


def listed():
    return [
        # a decode window of 8 rows between two layers: the experts' fp32 sum joins the residual
        _norm("norm_window", 8, 2048, x="fp32"),
        # a prompt chunk between two layers
        _norm("norm_chunk", 2048, 2048, x="fp32"),
        # several chunks at once in front of an 8-bit projection, a scale per 128 columns
        _norm("norm_8bit", 8192, 4096, out="e4m3", group=128),
        # one new token for 8 conversations
        _rope("rope_window", 8, 1, 4093, 16, 2),
        # a prompt chunk of 2,048 tokens in a context stretched to 32,768
        _rope("rope_prompt", 1, 2048, 32741, 32, 8, scaling="yarn", page=64, ragged=False),
        # prompts of different lengths, half of each head rotated, pairs side by side
        _rope("rope_ragged", 5, 901, 6011, 28, 4, rot=64, layout="interleaved", scaling="linear", page=32, dtype="fp16"),
        # the sampled token of one conversation, five alternatives
        _logprobs("logprobs_one", 1, 32000, 5, dtype="fp32"),
        # a decode window of 64 rows, an odd vocabulary, most of it ruled out by a grammar
        _logprobs("logprobs_window", 64, 50257, 20, masked=0.9, temperature=0.7),
        # every token of a prompt chunk scored
        _logprobs("logprobs_prompt", 2048, 131072, 1),
        # a full server's decode step: 64 states
        _linear("linear_step", "step", 64, 1, 16, 32),
        # one prompt chunk of 2,048 tokens
        _linear("linear_prompt", "chunk", 1, 2048, 16, 32, ragged=False),
        # eight prompts of different lengths
        _linear("linear_ragged", "chunk", 8, 4001, 16, 32),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["norm", "rope", "logprobs", "linear", "linear"])
    if op == "norm":
        H = rng.choice([2048, 4096, 512, _logint(rng, 64, 8192), 8 * _logint(rng, 8, 1024)])
        out = rng.choice(["bf16", "bf16", "fp16", "fp32", "e4m3"])
        group = rng.choice([0, 128, 32]) if out == "e4m3" and H % 128 == 0 else 0
        c = _norm("", _logint(rng, 1, min(65536, 8192 * 4096 // H)), H, rng.choice(["fp32", "bf16", "fp16"]),
                  rng.choice(["bf16", "fp16", "fp32"]), out, group)
    elif op == "rope":
        Hq, Hkv = rng.choice([(16, 4), (16, 2), (32, 8), (8, 8), (28, 4), (12, 4), (24, 1), (5, 5)])
        D = rng.choice([64, 128, 128, 80])
        B = _logint(rng, 1, 48)
        new = rng.choice([1, 1, 2, _logint(rng, 1, max(1, 2048 // B))])
        rot = rng.choice([D, D, D // 2, rng.randrange(2, D + 1, 2)])
        c = _rope("", B, new, _logint(rng, new, max(new, min(32741, 400000 // B))), Hq, Hkv, D, rot,
                  rng.choice(["half", "interleaved"]), rng.choice(["none", "linear", "yarn"]), rng.choice([16, 32, 64, 24]),
                  rng.choice(["bf16", "fp16"]), rng.random() < 0.7)
    elif op == "logprobs":
        V = _logint(rng, 257, 200000)
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        c = _logprobs("", _logint(rng, 1, min(4096, 2048 * 131072 * 2 // (V * SIZE[dtype]))), V,
                      rng.choice([0, 1, 5, 8, 20, 32]), dtype, rng.choice([0, 0, 1, 64]), rng.choice([0.0, 0.0, 0.9]),
                      rng.choice([1.0, 1.0, 0.7, 1.5]))
    else:
        Hk, Hv = rng.choice([(16, 32), (8, 8), (4, 16), (16, 16), (3, 6)])
        what = rng.choice(["step", "chunk"])
        if what == "step":
            c = _linear("", what, _logint(rng, 1, 64), rng.choice([1, 1, 1, 2, 3]), Hk, Hv)
        else:
            B = rng.choice([1, 1, 2, 5, 8])
            c = _linear("", what, B, _logint(rng, 2, min(4001, 20000 // B)), Hk, Hv, ragged=rng.random() < 0.7)
        c["D"], c["dtype"] = rng.choice([128, 128, 64]), rng.choice(["bf16", "bf16", "fp16"])
    c.pop("name")
    return c


def _spread(n, lo, hi):
    """n lengths over [lo, hi], the longest first, from a fixed low-discrepancy sequence."""
    return [hi if i == 0 else max(lo, int(lo + (hi - lo) * ((i * 0.6180339887498949) % 1.0))) for i in range(n)]


def _news(case):
    """New tokens per sequence."""
    if case.get("what") == "step" or case["new"] <= 3 or not case["ragged"]:
        return [case["new"]] * case["B"]
    return _spread(case["B"], max(1, case["new"] // 5), case["new"])


def _lens(case):
    """The sequences' lengths, new tokens included."""
    if not case["ragged"]:
        return [max(case["new"], case["max_len"])] * case["B"]
    return [max(n, x) for n, x in zip(_news(case), _spread(case["B"], max(1, case["max_len"] // 4), case["max_len"]))]


SIZE = {"bf16": 2, "fp16": 2, "fp32": 4, "e4m3": 1}


def work(case):
    if case["op"] == "norm":
        n, groups = case["T"] * case["H"], case["T"] * (case["H"] // case["group"] if case["group"] else 1)
        return {"bytes": n * (SIZE[case["x"]] + 2 * SIZE[case["res"]] + SIZE[case["out"]]) + 2 * case["H"]
                + (4 * groups if case["out"] == "e4m3" else 0), "flops": 5 * n}
    if case["op"] == "rope":
        T = sum(_news(case))
        return {"bytes": T * (2 * case["Hq"] + 4 * case["Hkv"]) * case["D"] * 2,
                "flops": 3 * T * (case["Hq"] + case["Hkv"]) * case["rot"]}
    if case["op"] == "logprobs":
        return {"bytes": case["T"] * (case["V"] * SIZE[case["dtype"]] + 8 * case["top"] + 24), "flops": 5 * case["T"] * case["V"]}
    T, D = sum(_news(case)), case["D"]
    state = 2 * 4 * case["B"] * case["Hv"] * D * D
    rows = T * (2 * case["Hk"] + 2 * case["Hv"]) * D * 2 + 4 * T * case["Hv"]
    # the recurrent form's operations: k v^T added to the decayed state, q S
    return {"bytes": state + rows, "flops": 5 * T * case["Hv"] * D * D}


# ------------------------------------------------------------------ inputs
def _frequencies(case):
    """Radians per token of each pair, and the factor on the rotated values."""
    rot, base = case["rot"], 10000.0
    f = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if case["scaling"] == "linear":
        return [x / 4.0 for x in f], 1.0
    if case["scaling"] == "yarn":  # a context of 8,192 stretched four times: long wavelengths by the factor, short ones not at all
        def pair_of(turns):
            return rot * math.log(8192 / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo, hi = max(math.floor(pair_of(32.0)), 0), min(math.ceil(pair_of(1.0)), rot - 1)
        ramp = [min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0) for i in range(rot // 2)]
        return [x * (1 - r) + x / 4.0 * r for x, r in zip(f, ramp)], 0.1 * math.log(4.0) + 1.0
    return f, 1.0


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed) * 7919 + 13)

    def randn(*shape, std=1.0, dtype="fp32"):
        return (torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32) * std).to(DTYPES[dtype])

    s = dict(case=case)
    if case["op"] == "norm":
        T, H = case["T"], case["H"]
        # a residual stream has a few columns that are far larger than the rest
        wide = torch.exp(torch.randn(H, generator=g, device=DEV))
        s["x"] = randn(T, H, dtype=case["x"])
        s["res"] = (randn(T, H) * wide).to(DTYPES[case["res"]])
        s["w"] = (1.0 + 0.2 * randn(H)).to(torch.bfloat16)
        s["out"] = torch.empty(T, H, dtype=E4M3 if case["out"] == "e4m3" else DTYPES[case["out"]], device=DEV)
        if case["out"] == "e4m3":
            s["scales"] = torch.empty(T, H // case["group"] if case["group"] else 1, dtype=torch.float32, device=DEV)
        return s
    if case["op"] == "logprobs":
        T, V, pad = case["T"], case["V"], case["pad"]
        z = torch.randn(T, V + pad, generator=g, device=DEV, dtype=torch.float32).mul_(2.5)
        best = torch.randint(0, V, (T, 8), generator=g, device=DEV)
        z.scatter_add_(1, best, 10 + 4 * torch.rand(T, 8, generator=g, device=DEV))
        if case["masked"]:
            z.masked_fill_(torch.rand(T, V + pad, generator=g, device=DEV) < case["masked"], -math.inf)
            z[:, 0] = 1.0  # a grammar always allows the end
        s["logits"] = z.to(DTYPES[case["dtype"]])[:, :V]
        # most tokens of a text are among the likely ones
        pick = torch.where(torch.rand(T, generator=g, device=DEV) < 0.8, best[:, 0], torch.randint(0, V, (T,), generator=g, device=DEV))
        s["tokens"] = pick.to(torch.int32)
        s["out"] = {n: torch.empty(T, dtype=dt, device=DEV) for n, dt in
                    (("logprob", torch.float32), ("rank", torch.int32), ("entropy", torch.float32))}
        if case["top"]:
            s["out"]["top_ids"] = torch.empty(T, case["top"], dtype=torch.int32, device=DEV)
            s["out"]["top_logprobs"] = torch.empty(T, case["top"], dtype=torch.float32, device=DEV)
        return s
    n_new = _news(case)
    T, B, D = sum(n_new), case["B"], case["D"]
    slots = torch.randperm(B, generator=g, device=DEV).to(torch.int32)
    # the i-th group of rows belongs to slot slots[i]; lengths and new tokens go by the slot
    new = torch.tensor(n_new, dtype=torch.int32, device=DEV)[slots.long()]
    s["slots"], s["row_start"] = slots, torch.cat([new.new_zeros(1), new.cumsum(0).to(torch.int32)])
    if case["op"] == "linear":
        Hk, Hv = case["Hk"], case["Hv"]
        qkv = randn(T, (2 * Hk + Hv), D, dtype=case["dtype"])  # parts of one projection
        qkv[:, :2 * Hk] = (qkv[:, :2 * Hk].float() * D ** -0.5).to(qkv.dtype)  # about unit keys and queries
        s["q"], s["k"], s["v"] = qkv[:, :Hk], qkv[:, Hk:2 * Hk], qkv[:, 2 * Hk:]
        # heads that remember from ten tokens to thousands, gated by the token
        rate = torch.exp(torch.linspace(math.log(1e-4), math.log(0.2), Hv, device=DEV))
        s["g"] = -(rate * torch.nn.functional.softplus(1.0 + randn(T, Hv)))
        s["state"] = randn(B, Hv, D, D)
        s["o"] = torch.empty(T, Hv, D, dtype=DTYPES[case["dtype"]], device=DEV)
        s["scale"] = 1.0
        return s
    page, Hkv, Hq, L = case["page"], case["Hkv"], case["Hq"], _lens(case)
    used = [-(-x // page) for x in L]
    n_pages, most = sum(used) + 3, max(used) + 1
    dt = DTYPES[case["dtype"]]
    s["k"] = torch.zeros(1, n_pages, Hkv, page, D, dtype=dt, device=DEV)
    s["v"] = torch.zeros_like(s["k"])
    order = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    s["table"] = torch.full((B, most), -1, dtype=torch.int32, device=DEV)
    s["refs"] = torch.zeros(n_pages, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(used):
        s["table"][b, :n] = order[at:at + n]
        at += n
    s["refs"][order[:at].long()] = 1
    s["lens"] = torch.tensor(L, dtype=torch.int32, device=DEV)
    s["free"] = torch.zeros(n_pages, dtype=torch.int32, device=DEV)
    s["free"][:n_pages - at] = order[at:]
    s["n_free"] = torch.full((1,), n_pages - at, dtype=torch.int32, device=DEV)
    qkv = randn(T, Hq + 2 * Hkv, D, dtype=case["dtype"])
    s["q"], s["k_new"], s["v_new"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    s["q_out"] = torch.empty(T, Hq, D, dtype=dt, device=DEV)
    f, s["gain"] = _frequencies(case)
    s["freq"] = torch.tensor(f, dtype=torch.float64, device=DEV)
    return s


# ------------------------------------------------------------------ the plain forms
def _plain_norm(s):
    case, wide = s["case"], torch.float64 if s["case"]["out"] == "e4m3" else torch.float32
    s["res"].copy_(s["x"].float() + s["res"].float())
    r = s["res"].to(wide)  # in 64 bits where e4m3's borders are near
    y = r * torch.rsqrt(r.square().mean(1, keepdim=True) + EPS) * s["w"].to(wide)
    if case["out"] != "e4m3":
        s["out"].copy_(y)
        return {"out": s["out"], "res": s["res"]}
    y = y.reshape(case["T"], s["scales"].shape[1], -1)
    scale = y.abs().amax(2, keepdim=True) / 448
    q = y / torch.where(scale == 0, torch.ones_like(scale), scale)
    s["out"].copy_(q.float().to(E4M3).reshape(case["T"], -1))
    s["scales"].copy_(scale[..., 0])
    return {"out": s["out"], "scales": s["scales"], "res": s["res"]}


def _places(s):
    """Of each row: its sequence, and its place among the sequence's rows."""
    start = s["row_start"].long()
    t = torch.arange(int(sum(_news(s["case"]))), device=DEV)
    b = (t[:, None] >= start[None, 1:]).sum(1)
    return b, t - start[b], start[1:] - start[:-1]


def _plain_rope(s):
    case = s["case"]
    rot, page = case["rot"], case["page"]
    b, i, n = _places(s)
    slot = s["slots"].long()
    pos = s["lens"][slot].long()[b] - n[b] + i
    a = pos.double()[:, None] * s["freq"][None]  # angles of far positions want 64 bits
    cos, sin = ((f(a) * s["gain"]).float()[:, None] for f in (torch.cos, torch.sin))

    def turned(x):
        x = x.float()
        if case["layout"] == "half":
            u, w = x[..., :rot // 2], x[..., rot // 2:rot]
            y = torch.cat([u * cos - w * sin, w * cos + u * sin], -1)
        else:
            u, w = x[..., 0:rot:2], x[..., 1:rot:2]
            y = torch.stack([u * cos - w * sin, w * cos + u * sin], -1).flatten(-2)
        return torch.cat([y, x[..., rot:]], -1).to(s["q"].dtype)

    pg = s["table"][slot[b], pos // page].long()
    s["k"][0, pg, :, pos % page] = turned(s["k_new"])
    s["v"][0, pg, :, pos % page] = s["v_new"]
    s["q_out"].copy_(turned(s["q"]))
    return {"q": s["q_out"], "k": s["k"], "v": s["v"]}


def _plain_logprobs(s):
    case = s["case"]
    raw = s["logits"].float()
    z = raw / case["temperature"]
    t = s["tokens"].long()[:, None]
    m = z.amax(1, keepdim=True)
    e = torch.exp(z - m)
    l = e.sum(1, keepdim=True)
    lse = m + torch.log(l)
    # a token that is ruled out adds nothing
    entropy = torch.log(l) - torch.where(e > 0, e * (z - m), torch.zeros_like(e)).sum(1, keepdim=True) / l
    mine = raw.gather(1, t)
    ids = torch.arange(case["V"], device=DEV)[None]
    rank = ((raw > mine) | ((raw == mine) & (ids < t))).sum(1)
    r = {"logprob": (z.gather(1, t) - lse)[:, 0], "rank": rank.int(), "entropy": entropy[:, 0]}
    if case["top"]:
        top = torch.sort(raw, dim=1, descending=True, stable=True)[1][:, :case["top"]]
        r["top_ids"], r["top_logprobs"] = top.int(), z.gather(1, top) - lse
    return r


BLOCK = 64


def _plain_linear(s):
    """Blocks of 64 tokens: each block's own sum of k v^T, the states between blocks as a
    decayed sum over the blocks before, and the products within a block."""
    case = s["case"]
    Hk, Hv, D, B = case["Hk"], case["Hv"], case["D"], case["B"]
    b, i, n = _places(s)
    Tm = -(-max(_news(case)) // BLOCK) * BLOCK
    nb, G = Tm // BLOCK, Hv // Hk
    slot = s["slots"].long()

    def padded(x, heads):  # -> [B][heads][blocks][BLOCK][..]
        y = torch.zeros(B, Tm, *x.shape[1:], dtype=torch.float32, device=DEV)
        y[b, i] = x.float()
        y = y.transpose(1, 2)
        return (y if heads == Hv else y.repeat_interleave(G, 1)).unflatten(2, (nb, BLOCK))

    q, k, v = padded(s["q"], Hk), padded(s["k"], Hk), padded(s["v"], Hv)
    g = padded(s["g"], Hv).double().cumsum(-1)            # [B][Hv][nb][BLOCK], within the block
    total = g[..., -1]
    before = total.cumsum(-1)                             # up to and with each block
    kv = torch.matmul((k * torch.exp(total[..., None] - g).float()[..., None]).transpose(-1, -2), v)
    # state in front of block c: the initial one, and block d's sum decayed over the blocks between
    c = torch.arange(nb + 1, device=DEV)
    ends = torch.cat([torch.zeros_like(before[..., :1]), before], -1)              # [B][Hv][nb + 1]
    w = torch.exp((ends[..., :, None] - ends[..., None, 1:]).masked_fill(c[:, None] <= c[None, :nb], -math.inf)).float()
    S0 = s["state"][slot]
    S = torch.matmul(w, kv.flatten(-2)) + torch.exp(ends).float()[..., None] * S0.flatten(-2)[:, :, None]
    S = S.unflatten(-1, (D, D))                                                     # [B][Hv][nb + 1][D][D]
    hide = torch.ones(BLOCK, BLOCK, dtype=torch.bool, device=DEV).triu(1)
    d = torch.exp((g[..., :, None] - g[..., None, :]).masked_fill(hide, -math.inf)).float()
    o = torch.matmul(torch.matmul(q, k.transpose(-1, -2)) * d, v)
    o += torch.matmul(q * torch.exp(g).float()[..., None], S[:, :, :nb])
    o = (o * s["scale"]).flatten(2, 3).transpose(1, 2)[b, i]                        # [T][Hv][D]
    s["o"].copy_(o)
    s["state"][slot] = S[:, :, nb]
    return {"o": s["o"], "state": s["state"]}


# ------------------------------------------------------------------ one pass
def _rotary(s):
    """The cache and the frequencies that a program keeps."""
    if "kv" not in s:
        from routed_expert_ffn_router_gb300.block import Rotary
        from routed_expert_ffn_router_gb300.paged import PagedKV
        case = s["case"]
        scaling = {"none": None, "linear": dict(kind="linear", factor=4.0),
                   "yarn": dict(kind="yarn", factor=4.0, original=8192)}[case["scaling"]]
        s["rotary"] = Rotary(case["rot"], base=10000.0, layout=case["layout"], scaling=scaling, device=DEV)
        s["kv"] = PagedKV.over(s["k"], s["v"], s["table"], s["lens"], s["refs"], s["free"], s["n_free"], Hq=case["Hq"],
                               max_rows=0)
    return s["kv"], s["rotary"]


def _states(s):
    if "layer" not in s:
        from routed_expert_ffn_router_gb300.linear import LinearAttention
        s["layer"] = LinearAttention.over(s["state"], s["case"]["Hk"], dtype=s["q"].dtype)
    return s["layer"]


def run(s):
    case = s["case"]
    if not own:
        return {"norm": _plain_norm, "rope": _plain_rope, "logprobs": _plain_logprobs, "linear": _plain_linear}[case["op"]](s)
    if case["op"] == "norm":
        from routed_expert_ffn_router_gb300.block import rms_norm
        if case["out"] == "e4m3":
            rms_norm(s["x"], s["w"], residual=s["res"], eps=EPS, group=case["group"], out=s["out"], scales=s["scales"])
            return {"out": s["out"], "scales": s["scales"], "res": s["res"]}
        rms_norm(s["x"], s["w"], residual=s["res"], eps=EPS, out=s["out"])
        return {"out": s["out"], "res": s["res"]}
    if case["op"] == "rope":
        kv, rotary = _rotary(s)
        q = kv.append_rotary(0, s["q"], s["k_new"], s["v_new"], rotary, slots=s["slots"], row_start=s["row_start"],
                             q_out=s["q_out"])
        return {"q": q, "k": s["k"], "v": s["v"]}
    if case["op"] == "logprobs":
        from routed_expert_ffn_router_gb300.block import token_logprobs
        return token_logprobs(s["logits"], s["tokens"], top=case["top"], temperature=case["temperature"],
                              out=s["out"])
    layer = _states(s)
    if case["what"] == "step":
        layer.step(s["q"], s["k"], s["v"], s["g"], slots=s["slots"], scale=s["scale"], out=s["o"])
    else:
        layer.chunk(s["q"], s["k"], s["v"], s["g"], slots=s["slots"], row_start=s["row_start"], scale=s["scale"], out=s["o"])
    return {"o": s["o"], "state": s["state"]}


# ------------------------------------------------------------------ the definition, in 64 bits
def _exact_norm(s):
    case = s["case"]
    r = (s["x"].float() + s["res"].float()).to(s["res"].dtype).double()  # what the residual holds is what is normed
    root = torch.sqrt((r * r).sum(1) / case["H"] + EPS)
    y = r / root[:, None] * s["w"].double()[None]
    if case["out"] != "e4m3":
        return {"out": y, "res": r}
    width = case["group"] or case["H"]
    top = y.abs().reshape(case["T"], -1, width).max(2)[0]
    return {"out": y / (top / 448).clamp(min=1e-300).repeat_interleave(width, 1), "scales": top / 448, "res": r}


def _exact_rope(s):
    case, dev = s["case"], DEV
    rot, page, start = case["rot"], case["page"], s["row_start"].tolist()
    freq, gain = _frequencies(case)
    freq = torch.tensor(freq, dtype=torch.float64, device=dev)
    first = list(range(rot // 2)) if case["layout"] == "half" else list(range(0, rot, 2))
    second = list(range(rot // 2, rot)) if case["layout"] == "half" else list(range(1, rot, 2))
    q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
    k_new, v_new = s["k_new"].double(), s["v_new"].double()
    for b, slot in enumerate(s["slots"].tolist()):
        L, n = int(s["lens"][slot]), start[b + 1] - start[b]
        pos = torch.arange(L - n, L, device=dev)
        turn = torch.polar(torch.full((n, rot // 2), gain, dtype=torch.float64, device=dev), pos.double()[:, None] * freq)
        for x in (q, k_new):
            part = x[start[b]:start[b + 1]]
            z = torch.complex(part[..., first], part[..., second]) * turn[:, None]
            part[..., first], part[..., second] = z.real, z.imag
        pages = s["table"][slot].long()[pos // page]
        k[0, pages, :, pos % page] = k_new[start[b]:start[b + 1]]
        v[0, pages, :, pos % page] = v_new[start[b]:start[b + 1]]
    return {"q": q, "k": k, "v": v}


def _exact_logprobs(s):
    case = s["case"]
    r = {"logprob": [], "rank": [], "entropy": [], "top_ids": [], "top_logprobs": []}
    for z0, t in zip(s["logits"].split(64), s["tokens"].long().split(64)):
        z = z0.double() / case["temperature"]
        lp = z - torch.logsumexp(z, 1, keepdim=True)
        mine = lp.gather(1, t[:, None])
        r["logprob"].append(mine[:, 0])
        r["entropy"].append(-torch.xlogy(lp.exp(), lp.exp()).sum(1))
        order = torch.sort(z0.double(), dim=1, descending=True, stable=True)[1]
        r["rank"].append((order == t[:, None]).int().argmax(1).int())
        r["top_ids"].append(order[:, :case["top"]].int())
        r["top_logprobs"].append(lp.gather(1, order[:, :case["top"]]))
    r = {name: torch.cat(x) for name, x in r.items()}
    if not case["top"]:
        r.pop("top_ids"), r.pop("top_logprobs")
    return r


def _exact_linear(s):
    """Token by token, all sequences and heads at once."""
    case = s["case"]
    G, start, slots = case["Hv"] // case["Hk"], s["row_start"].tolist(), s["slots"].tolist()
    S, o = s["state"].double(), torch.zeros(s["o"].shape, dtype=torch.float64, device=DEV)
    news = [b - a for a, b in zip(start, start[1:])]
    q, k = (s[n].double().repeat_interleave(G, 1) for n in ("q", "k"))
    v, decay = s["v"].double(), torch.exp(s["g"].double())
    for i in range(max(news)):
        live = [b for b, n in enumerate(news) if n > i]
        at = torch.tensor([start[b] + i for b in live], device=DEV)
        sl = torch.tensor([slots[b] for b in live], device=DEV)
        S[sl] = S[sl] * decay[at][..., None, None] + k[at][..., None] * v[at][..., None, :]
        o[at] = (q[at][..., None, :] @ S[sl])[..., 0, :] * s["scale"]
    return {"o": o, "state": S}


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "rope": _exact_rope, "logprobs": _exact_logprobs, "linear": _exact_linear}[case["op"]](s)

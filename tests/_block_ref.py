"""Plain 64-bit references of the decoder-block operators (test infrastructure
only). Tolerances are counted from roundings: u is half a step of a 16-bit type,
F = 2^-24 half a step of fp32."""
import math

import torch

F = 2.0 ** -24
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25, torch.float32: 0.0}  # half a step below the normal range


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def norm(x, w, res, eps, w_offset, out_dtype):
    """-> (residual as it is then held, y and its tolerance in float64). Per row: up to 64
    squares added per thread and a tree of ten, so 40 F of the root; then the root, the
    quotient and two products: 48 F in all with a margin of 2; one rounding."""
    if res is not None:
        res = (x.float() + res.float()).to(res.dtype)
    r = (x if res is None else res).double()
    y = r / torch.sqrt(r.square().mean(1, keepdim=True) + eps)
    if w is not None:
        y = y * (w.double() + w_offset)
    u = half_step(out_dtype) if out_dtype in TINY else 0.0
    return res, y, y.abs() * (u + 96 * F) + TINY.get(out_dtype, 0.0) + 1e-44


def turned(x, pos, freq, gain, rot, layout):
    """x [rows][heads][D] in float64 turned by pos [rows] * freq; tolerance of its fp32
    form before the last rounding: the angle is off by 2^-25 half turns (its conversion
    to fp32) and 2^-32, sine and cosine by 2 F, their gain and the two products and the
    sum by 5 F: 16 F of |x| + |y| with a margin."""
    x = x.double()
    half = rot // 2
    i0 = torch.arange(half) if layout == "half" else torch.arange(half) * 2
    i1 = i0 + (half if layout == "half" else 1)
    a = pos.double()[:, None] * torch.tensor(freq, dtype=torch.float64, device=x.device)[None]
    c, s = (torch.cos(a) * gain)[:, None], (torch.sin(a) * gain)[:, None]
    y, tol = x.clone(), torch.zeros_like(x)
    u, v = x[..., i0], x[..., i1]
    y[..., i0], y[..., i1] = u * c - v * s, v * c + u * s
    tol[..., i0] = tol[..., i1] = (u.abs() + v.abs()) * abs(gain) * 16 * F
    return y, tol


def logprobs(z, tokens, top, temperature, threads=512):
    """-> dict of float64 and whole numbers, and their tolerances. A logit's distance to the
    maximum carries one rounding and its quotient another: 2 F |d|; an exponential is
    off by that of its argument (twice, in base 2) and 4 F; a lane adds up to V / threads
    of them before a tree of 14."""
    zd = z.double()
    T, V = z.shape
    m = zd.amax(1, keepdim=True)
    d = torch.where(zd == m, torch.zeros_like(zd), (zd - m)) / temperature
    e = torch.exp(d)
    l = e.sum(1, keepdim=True)
    p = e / l
    pd = torch.where(e > 0, p * d, torch.zeros_like(d))
    ln_l, mean_d = torch.log(l), pd.sum(1)
    lp = d - ln_l
    ent = ln_l[:, 0] - mean_d
    far = (V / threads + 60) * F + 6 * F * mean_d.abs()                  # of ln l, relative to l
    pd2 = torch.where(e > 0, p * d * d, torch.zeros_like(d)).sum(1)      # a term's own share: d may be off by 2 F |d|
    r = {"entropy": ent}
    tol = {"entropy": far * (2 + mean_d.abs() * 2) + 8 * F * pd2 + 4 * F * ent.abs() + 8 * F * ln_l[:, 0].abs()}

    def tol_of(x):  # x: logarithms, [T][n]
        big = x + ln_l
        return torch.where(torch.isfinite(x), 4 * F * big.abs().nan_to_num(0, 0, 0) + far[:, None] + 4 * F * ln_l.abs()
                           + 2 * F * x.abs().nan_to_num(0, 0, 0), torch.zeros_like(x))
    order = torch.sort(torch.where(torch.isnan(z), torch.full_like(z, -math.inf), z).float(), dim=1, descending=True, stable=True)[1]
    if tokens is not None:
        t = tokens.long()
        has = (t >= 0) & (t < V)
        mine = lp.gather(1, t.clamp(0, V - 1)[:, None])
        r["logprob"] = torch.where(has, mine[:, 0], torch.zeros_like(mine[:, 0]))
        tol["logprob"] = tol_of(mine)[:, 0]
        r["rank"] = torch.where(has, (order == t[:, None]).int().argmax(1).int(), -1).int()
    if top:
        r["top_ids"] = order[:, :top].int()
        r["top_logprobs"] = lp.gather(1, order[:, :top])
        tol["top_logprobs"] = tol_of(r["top_logprobs"])
    return r, tol


def linear(q, k, v, g, state, spans, scale, matrix=False):
    """Token by token in float64. spans: (slot, first row, rows). -> o, its tolerance,
    state, its tolerance. With A the same recurrence over magnitudes, a token costs
    the state a rounding of its decay (4 F), of the product and of the sum: 6 F; o adds
    Dk products. matrix: products on the tensor cores, in which a score and a state
    enter rounded once to the type (u each of their term) and a decayed key or value as
    two values of the type (4 u^2); sums of up to 128 + Dk terms that may truncate (2 F each)."""
    u = half_step(q.dtype)
    G = v.shape[1] // k.shape[1]
    kd, qd = (x.double().repeat_interleave(G, 1) for x in (k, q))
    vd = v.double()
    gd = g.double().clamp(max=0).expand(q.shape[0], v.shape[1])
    S, o = state.double().clone(), torch.zeros(v.shape, dtype=torch.float64, device=v.device)
    tS, to = torch.zeros_like(S), torch.zeros_like(o)
    Dk = q.shape[2]
    for slot, r0, n in spans:
        A = S[slot].abs()
        for t in range(r0, r0 + n):
            e = torch.exp(gd[t])[:, None, None]
            S[slot] = S[slot] * e + kd[t][:, :, None] * vd[t][:, None, :]
            A = A * e + (kd[t][:, :, None] * vd[t][:, None, :]).abs()
            o[t] = (qd[t][:, None] @ S[slot])[:, 0] * scale
            part = (qd[t].abs()[:, None] @ A)[:, 0] * abs(scale)
            i = t - r0 + 1
            to[t] = u * o[t].abs() + part * ((Dk + 8 + 6 * i) * F + ((2 * u + 4 * u * u + 2 * (128 + Dk) * F) if matrix else 0)) \
                + TINY[q.dtype] + 1e-30
        tS[slot] = A * ((8 + 6 * n) * F + ((4 * u * u + 2 * 128 * F) if matrix else 0)) + 1e-30
    return o, to, S, tS


def within(got, want, tol, what=""):
    """got and want agree to tol; infinities and NaN in the same places."""
    g, w = got.double(), want.double()
    bad = torch.isnan(w) != torch.isnan(g)
    inf = torch.isinf(w) | torch.isinf(g)
    bad |= inf & (g != w) & ~torch.isnan(w)
    fin = torch.isfinite(w) & torch.isfinite(g)
    off = torch.where(fin, (g - w).abs() - tol, torch.zeros_like(g))
    bad |= off > 0
    if bad.any():
        i = tuple(x[0].item() for x in bad.nonzero(as_tuple=True))
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {i}: got {g[i].item()!r}, "
                             f"want {w[i].item()!r} +- {torch.as_tensor(tol).expand_as(g)[i].item():.3e}")

"""The state of a prompt chunk in 64 bits with a tight bound (test infrastructure only):
for keys of which few in a block of 128 tokens are not zero, the sums in the tensor
cores have few terms and what is left is the rounding of each."""
import math

import torch

F = 2.0 ** -24  # half a step of fp32
BLOCK = 128


def state(k, v, g, state0, spans, terms, two_values=False):
    """Token by token in float64. spans: (slot, first row, rows); terms: tokens of a block
    with a key, no two of them in the same 16. -> state, its bound. With A the recurrence over
    magnitudes, in units of F:
      a decay's exponent is a difference of sums of logarithms (to base 2) that are held as
      pairs: two roundings of it, so 2 |g| log2 e per token over which a term decays;
      the exponential 4, its product with the key 1; in fp16 the key as two values of the
      type: 2^-22 of it, so 4 (in bf16 three values are all of it);
      a term enters as up to three products, exact each; each sum of the accumulator is
      off by up to 2 of its magnitudes: 6 `terms`;
      a block's end: the factor e^G 4 and two sums, and once more where the CTAs of a
      cluster put their parts together: 12.
    In fp16 besides, not relative to a term: the block's largest |k| is brought to 2^13 or
    more, and what enters, the key decayed to the block's END times that factor, is off by
    half the type's smallest step: 2^-25, so 2^-38 of the largest |k|. It is the decayed key
    that is rounded, so this stands at the block's end as it is, however far the key itself
    has decayed by then: sum over the block's terms of 2^-38 max|k| |v|, added there.
    two_values: the keys in bf16 as two values, cut, which the bound has to show."""
    bits16, G = k.dtype == torch.float16, v.shape[1] // k.shape[1]
    kd, vd = k.double().repeat_interleave(G, 1), v.double()
    gd = g.double().clamp(max=0)
    S, tol = state0.double().clone(), torch.zeros(state0.shape, dtype=torch.float64, device=state0.device)
    each = (9 if bits16 else 5) + 6 * terms
    for slot, r0, n in spans:
        A, tS = S[slot].abs(), torch.zeros_like(S[slot])
        for b0 in range(r0, r0 + n, BLOCK):
            b1 = min(b0 + BLOCK, r0 + n)
            low = 2.0 ** -38 * float(kd[b0:b1].abs().max()) if bits16 else 0.0
            floor = torch.zeros_like(vd[r0])
            for t in range(b0, b1):
                e = torch.exp(gd[t])[:, None, None]
                turns = torch.where(e > 0, -gd[t][:, None, None] * math.log2(math.e), torch.zeros_like(e))
                tS = (tS + 2 * F * turns * A) * e
                if not kd[t].any():
                    S[slot] = S[slot] * e
                    A = A * e
                    continue
                kt = kd[t]
                if two_values:
                    rest = torch.exp(gd[t + 1:b1].sum(0))[:, None]
                    kt = _cut16(kt * rest) / rest
                x = kt[:, :, None] * vd[t][:, None, :]
                S[slot] = S[slot] * e + x
                A = A * e + x.abs()
                tS = tS + each * F * x.abs()
                floor = floor + low * vd[t].abs()
            tS = tS + 12 * F * A + floor[:, None, :]
        tol[slot] = tS + 1e-30
    return S, tol


def _cut16(x):
    """The upper 16 of an fp32's 24 bits, as two values of 8 hold them."""
    return (x.float().view(torch.int32) & -256).view(torch.float32).double()

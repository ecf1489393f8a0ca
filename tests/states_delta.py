"""dK of the few-rows backward in 64 bits, with a bound that follows the kernel's rule for delta.

delta comes from the rounded output, so a row's is off by c = sum dO (O rounded - O), which the output that the call was
given tells exactly.  A state with a weight of `large` or more in some row is noted, and computed with delta from sums in
32 bits; the others' dS keeps p c.  Beside that, of dS: two roundings of the 16-bit halves (u^2), p's relative error r
(2 es + 2^-20 + e |s|, es that of a score's sum; also through a corrected delta), and the 32-bit sums of dP, of delta and
of the row (e (d + 4) and e n of their terms).  And dK's own rounding, u, and its sum over the rows.
"""

import torch

import states_reference as ref


def large_weight(rows):
    """The weight from which a state is noted, by the packed rows of the call's longest item."""
    return 0.125 if rows <= 8 else 0.25


def item(q, k, v, d_o, o, scale, large, dtype, noted=None):
    """(dK, its bound, what a kernel with this rule gives before dK's rounding) of one item and key head: q, d_o and the
    rounded output o [rows, d], k and v [states, d], all in 64 bits.  `noted` overrides the rule for the last one."""
    u, e, tiny = ref.UNIT[dtype], ref.E, ref.TINY[dtype]
    d, n = q.shape[1], k.shape[0]
    s = scale * q @ k.T
    p = s.softmax(-1)
    dp = d_o @ v.T
    exact = p @ v
    delta = (d_o * exact).sum(-1, keepdim=True)
    c = (d_o * (o - exact)).sum(-1, keepdim=True)
    ds = p * (dp - delta)
    es = (d + 4) * e * scale * (q.abs() @ k.abs().T).amax(-1, keepdim=True)
    r = 2 * es + 2.0 ** -20 + e * s.abs().amax(-1, keepdim=True)
    mag = d_o.abs() @ v.abs().T
    sums = (d + 4) * e * (d_o.abs() * o.abs()).sum(-1, keepdim=True)
    row = (r * ds.abs() + (d + 4) * e * p * mag + n * e * (ds.abs() + p * c.abs())).sum(-1, keepdim=True) + r * c.abs()
    # a weight within its own error of the limit may go either way
    kept_error = p.amax(0) < large * (1 + 2 * r.amax())
    b = (u * u + r) * ds.abs() + tiny + p * ((d + 4) * e * mag + torch.where(kept_error, c.abs() + sums, row))
    want = scale * ds.T @ q
    bound = (u + 2.0 ** -20) * want.abs() + scale * (b + (q.shape[0] + 4) * e * ds.abs()).T @ q.abs() + tiny
    off = ~(p.amax(0) >= large) if noted is None else ~noted(p)
    return want, bound, scale * (p * (dp - delta - torch.where(off, c, 0.0))).T @ q


CASES = [
    # packed rows of an item and key head, states of the items, head dimension
    (1, [700, 90, 300, 1000] * 6, 128), (8, [300, 64, 1500] * 4, 64), (12, [700, 333] * 6, 72), (16, [900, 200, 40] * 4, 128),
]

"""The token-state operators in 64 bits, written from their formulas, with bounds on the rounding error of a kernel that
computes in 32 bits, feeds its matrix products operands of the inputs' type and rounds once at the end.

Bounds, element by element, with u the unit roundoff of the type (2^-8 bf16, 2^-11 fp16, 2^-24 fp32) and e = 2^-24:
  rotation   u |y| + 4 e (|x_a c| + |x_b s|): two products and a sum
  norm       the same on the normalised values, whose factor 1/sqrt(mean + epsilon) is a sum of D squares (D e relative
             at most, halved by the square root) and a reciprocal square root to 4 e
  attention  a score is a sum of D products in 32 bits: it is off by at most es = (D + 4) e scale sum|q k|, so an
             exponential by 2 es + 2^-20 relative (the row's maximum or lse is off by as much; 2^-20 covers the
             exponential itself, its argument's rounding where |s| < 16, and sums).  P as an operand: u relative, or
             half the type's smallest subnormal.
"""

import numpy as np
import torch

E = 2.0 ** -24
UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}   # half the smallest subnormal


def table(positions, rotary_dim, base=10000.0):
    i = np.arange(rotary_dim // 2)
    a = np.arange(positions)[:, None] * base ** (-2.0 * i / rotary_dim)
    return torch.from_numpy(np.stack([np.cos(a), np.sin(a)], axis=-1).astype(np.float32))


def pairs(rotary_dim, interleaved):
    a = torch.arange(0, rotary_dim, 2) if interleaved else torch.arange(rotary_dim // 2)
    return a, a + 1 if interleaved else a + rotary_dim // 2


def rotate(x, tab, positions, interleaved, back=False):
    """(rotated, bound of |products|) of x [rows, heads, dim] in 64 bits."""
    a, b = pairs(2 * tab.shape[1], interleaved)
    cs = tab.double()[positions]
    c, s = cs[:, None, :, 0], cs[:, None, :, 1] * (-1 if back else 1)
    y, m = x.clone(), x.abs()
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    m[..., a] = (x[..., a] * c).abs() + (x[..., b] * s).abs()
    m[..., b] = (x[..., b] * c).abs() + (x[..., a] * s).abs()
    return y, m


def norm_rotate(x, gain, tab, positions, interleaved, epsilon):
    r = (x.pow(2).mean(-1, keepdim=True) + epsilon).rsqrt()
    return rotate(x * r * gain, tab, positions, interleaved)


def norm_rotate_backward(x, dy, gain, tab, positions, interleaved, epsilon):
    """(dx, bound of |terms|, d_gain, bound of |terms|)."""
    d = x.shape[-1]
    r = (x.pow(2).mean(-1, keepdim=True) + epsilon).rsqrt()
    n = x * r
    dz, mz = rotate(dy, tab, positions, interleaved, back=True)
    t = dz * gain
    dx = r * (t - n * (t * n).mean(-1, keepdim=True))
    m = r * ((mz * gain).abs() + n.abs() * (mz * gain * n).abs().sum(-1, keepdim=True) / d)
    return dx, m, (dz * n).sum((0, 1)), (mz * n.abs()).sum((0, 1))


def attention(q, k, v, q_len, k_len, scale, mask=None, d_o=None, shared=False, dtype=torch.bfloat16):
    """Outputs, gradients (with d_o) and their bounds, in 64 bits: dict of name -> (value, bound).  q [rows, heads, dim],
    k and v [states, key_heads, dim]; q_len None: the queries are every item's (shared)."""
    u, tiny = UNIT[dtype], TINY[dtype]
    rows, hq, d = q.shape
    hk = k.shape[1]
    g = hq // hk
    items = len(k_len)
    out_rows = rows * items if shared else rows
    z = lambda n, h: torch.zeros(n, h, d, dtype=torch.float64, device=q.device)  # noqa: E731
    res = {"output": (z(out_rows, hq), z(out_rows, hq)), "d_q": (z(rows, hq), z(rows, hq)),
           "d_k": (z(k.shape[0], hk), z(k.shape[0], hk)), "d_v": (z(k.shape[0], hk), z(k.shape[0], hk))}
    lse = torch.full((out_rows, hq), -float("inf"), dtype=torch.float64, device=q.device)
    lse_b = torch.zeros_like(lse)
    q0 = k0 = o0 = 0
    for i in range(items):
        nq, nk = rows if shared else q_len[i], k_len[i]
        keep = torch.arange(k0, k0 + nk, device=q.device)
        if mask is not None:
            keep = keep[mask[k0:k0 + nk] != 0]
        if keep.numel() and nq:
            Q = q[q0:q0 + nq].double().reshape(nq, hk, g, d)
            K, V = k[keep].double(), v[keep].double()
            S = scale * torch.einsum("rhgd,khd->hgrk", Q, K)
            es = (d + 4) * E * abs(scale) * torch.einsum("rhgd,khd->hgrk", Q.abs(), K.abs()).amax(-1, keepdim=True)
            rel = 2 * es + 2.0 ** -20 + E * S.abs().amax(-1, keepdim=True)
            L = torch.logsumexp(S, -1)
            P = torch.exp(S - L[..., None])
            top = P.amax(-1, keepdim=True)
            O = torch.einsum("hgrk,khd->rhgd", P, V)
            # the forward's operand is P over the row's largest, times 2^8 at most
            bP = P * (rel + u) + tiny * top
            A = torch.einsum("hgrk,khd->rhgd", bP, V.abs())
            res["output"][0][o0:o0 + nq] = O.reshape(nq, hq, d)
            res["output"][1][o0:o0 + nq] = (A + u * O.abs() + tiny).reshape(nq, hq, d)
            lse[o0:o0 + nq] = L.permute(2, 0, 1).reshape(nq, hq)
            lse_b[o0:o0 + nq] = (es + 2.0 ** -20 + 4 * E * L.abs()[..., None])[..., 0].permute(2, 0, 1).reshape(nq, hq)
            if d_o is not None:
                dO = d_o[o0:o0 + nq].double().reshape(nq, hk, g, d)
                dP = torch.einsum("rhgd,khd->hgrk", dO, V)
                delta = (P * dP).sum(-1, keepdim=True)
                dS = P * (dP - delta)
                mag = torch.einsum("rhgd,khd->hgrk", dO.abs(), V.abs())
                # the row sum of dO * O from the rounded output
                b_delta = torch.einsum("rhgd,rhgd->hgr", dO.abs(), (A + (u + d * E) * O.abs()).reshape(nq, hk, g, d))
                bP = P * (rel + u) + tiny
                bS = dS.abs() * (rel + u) + P * (b_delta[..., None] + (d + 4) * E * mag) + tiny
                dV = torch.einsum("hgrk,rhgd->khd", P, dO)
                bV = torch.einsum("hgrk,rhgd->khd", bP, dO.abs())
                dQ = scale * torch.einsum("hgrk,khd->rhgd", dS, K)
                bQ = abs(scale) * torch.einsum("hgrk,khd->rhgd", bS, K.abs())
                dK = scale * torch.einsum("hgrk,rhgd->khd", dS, Q)
                bK = abs(scale) * torch.einsum("hgrk,rhgd->khd", bS, Q.abs())
                res["d_v"][0][keep], res["d_v"][1][keep] = dV, bV
                res["d_k"][0][keep], res["d_k"][1][keep] = dK, bK
                res["d_q"][0][q0:q0 + nq] += dQ.reshape(nq, hq, d)
                res["d_q"][1][q0:q0 + nq] += bQ.reshape(nq, hq, d)
        k0 += nk
        o0 += nq
        if not shared:
            q0 += nq
    for name in ("d_q", "d_k", "d_v"):
        val, b = res[name]
        res[name] = (val, b + u * val.abs() + 2.0 ** -20 * val.abs() + tiny)
    res["lse"] = (lse, lse_b)
    return res

"""The operators between a tower's blocks in 64 bits, plainly, each result with a bound on the error of 32-bit arithmetic.

The bounds count roundings, U = 2^-24 each (half an ulp of fp32, relative to the value).  A sum over a row runs through at
most 70 additions in series (32 in a thread, 5 across a warp's lanes, 32 across warps) and is off by 70 U of the sum of
magnitudes.  With c = z - mean, s^2 = mean c^2, r = 1 / sqrt(s^2 + epsilon) and n = c r:

  deviations   the mean is off by 70 U mean|z|; d = z - m is exact but for U |d|, and subtracting its own mean e leaves c
               but for 2 U |c| + 76 U s, where |e| <= s / 4: rows whose mean is below 6e4 times their spread;
  variance     off by 120 U s^2, so r by 60 U, and 5 U for the square root's reciprocal (2 ulp) and its argument;
  n            off by U (75 |n| + 80), as r s <= 1;
  gradient     with t = gain d_y, A = mean|t|, B = mean|t n|: mean t is off by 71 U A, mean(t n) by U (145 B + 112 A), and
               r (t - mean t - n mean(t n)) by r U (75 |t| + 145 A + 80 B + |n| (300 B + 115 A));
  sums over rows   each term by |d_y| times n's error, the sum by (rows + 100) U of the terms' magnitudes.

Where the input of the norm is itself a rounded sum, off by dz, n moves by r (dz + mean dz) + |n| r rms(dz).
A result rounded to its type is off by another half step, eps / 2 of the value, or half of the smallest number.
"""

import torch

U = 2.0 ** -24


def rounded(value, error, dtype):
    """(value, bound) of a result computed to within `error` and rounded to dtype."""
    f = torch.finfo(dtype)
    half = f.eps / 2
    return value, error * (1 + half) + half * value.abs() + f.smallest_normal * half


def words(rows, width, seed, step, site):
    """The generator's words, [rows, width]: whole numbers in Python's arithmetic, one block at a time."""
    low, out = 2 ** 32 - 1, torch.empty(rows, (width + 3) // 4 * 4, dtype=torch.int64)
    for r in range(rows):
        for k in range((width + 3) // 4):
            out[r, 4 * k:4 * k + 4] = torch.tensor(philox([k + 65536 * site, r, step & low, step >> 32], [seed & low, seed >> 32]))
    return out[:, :width]


def philox(c, k):
    c, k = list(c), list(k)
    for _ in range(10):
        p, q = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(q >> 32) ^ c[1] ^ k[0], q & (2 ** 32 - 1), (p >> 32) ^ c[3] ^ k[1], p & (2 ** 32 - 1)]
        k = [(k[0] + 0x9E3779B9) % 2 ** 32, (k[1] + 0xBB67AE85) % 2 ** 32]
    return c


def factors(rows, width, rate, seed, step, site):
    """[rows, width]: 0, or the inverse of the share that is kept."""
    drop = int(rate * 2.0 ** 32)
    return (words(rows, width, seed, step, site) >= drop).double() * (2.0 ** 32 / (2.0 ** 32 - drop))


def dropout(x, factor, dtype):
    y = torch.where(factor == 0, 0.0, x.double() * factor)
    return rounded(y, 2 * U * y.abs(), dtype)


def mean(x):
    return x.mean(dim=1, keepdim=True)


def statistics(z, epsilon):
    c = z - mean(z)
    r = 1 / torch.sqrt(mean(c * c) + epsilon)
    return c * r, r


def layer_norm(x, gain, bias, epsilon, dtype, off=None):
    """`off`: the error of x, where it is itself computed."""
    z = x.double()
    n, r = statistics(z, epsilon)
    n_off = U * (75 * n.abs() + 80)
    if off is not None:
        n_off = n_off + r * (off + mean(off)) + n.abs() * r * mean(off * off).sqrt()
    y = n * gain.double() + bias.double()
    return rounded(y, gain.double().abs() * n_off + 2 * U * y.abs() + U * (n * gain).abs(), dtype)


def layer_norm_backward(x, d_y, gain, epsilon, dtype):
    """d_x (of the stream's type), d_gain, d_bias, and the 64-bit d_x with its error before it is rounded."""
    z, g, w = x.double(), d_y.double(), gain.double()
    n, r = statistics(z, epsilon)
    t = g * w
    d = r * (t - mean(t) - n * mean(t * n))
    a, b = mean(t.abs()), mean((t * n).abs())
    off = r * U * (75 * t.abs() + 145 * a + 80 * b + n.abs() * (300 * b + 115 * a))
    rows = z.shape[0]

    def summed(terms, each):
        return rounded(terms.sum(0), each.sum(0) + (rows + 100) * U * terms.abs().sum(0), torch.float32)
    return {"d_x": rounded(d, off, dtype), "d_gain": summed(g * n, g.abs() * U * (75 * n.abs() + 80)),
            "d_bias": summed(g, torch.zeros_like(g)), "plain": (d, off)}


def join(x, residual, factor, gain, bias, epsilon):
    xs = torch.where(factor == 0, 0.0, x.double() * factor)
    z = residual.double() + xs
    off = U * (2 * xs.abs() + z.abs())
    return {"sum": rounded(z, off, residual.dtype), "output": layer_norm(z, gain, bias, epsilon, x.dtype, off)}


def join_backward(total, d_y, d_sum, factor, gain, epsilon):
    b = layer_norm_backward(total, d_y, gain, epsilon, total.dtype)
    d, off = b["plain"]
    if d_sum is not None:
        d = d + d_sum.double()
        off = off + 2 * U * d.abs()
    dx = torch.where(factor == 0, 0.0, d * factor)
    return {"d_residual": rounded(d, off, total.dtype), "d_x": rounded(dx, off * factor + 3 * U * dx.abs(), d_y.dtype),
            "d_gain": b["d_gain"], "d_bias": b["d_bias"]}

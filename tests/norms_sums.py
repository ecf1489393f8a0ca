"""Bounds on the gains' and biases' gradients by the additions that the kernels' sums over rows have in series: norms_reference
allows as many as there are rows, which hides a lost row once there are some thousands."""

import torch

import norms_reference as ref


def depth(rows, sms):
    """Additions in series of a sum over rows, at most.  Of B blocks of T teams each team takes rows / (B T) rows and one more;
    a block adds T teams' sums, a warp of the second kernel B / 32 blocks' and that one 32 warps'.  B is the number of SMs at
    least (or a team takes one row), and at most four times that; T is 128 at most.  So a team's and a block's are
    rows / (SMs T) + 2 + T, which is largest at T = 1 or at T = 128.  One block, which 256 rows at most have to themselves,
    adds no more."""
    return 256 if rows <= 256 else max(rows // sms + 3, rows // (128 * sms) + 130) + sms // 8 + 1 + 32


def summed(terms, each, sms):
    """(value, bound) of a sum over rows, each term computed to within `each`."""
    return ref.rounded(terms.sum(0), each.sum(0) + depth(len(terms), sms) * ref.U * terms.abs().sum(0), torch.float32)


def gradient_sums(z, d_y, sms, epsilon=1e-5):
    n, _ = ref.statistics(z.double(), epsilon)
    g = d_y.double()
    return {"d_gain": summed(g * n, g.abs() * ref.U * (75 * n.abs() + 80), sms), "d_bias": summed(g, torch.zeros_like(g), sms)}

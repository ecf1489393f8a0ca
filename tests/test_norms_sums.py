"""The bounds of tests/norms_sums.py on the CPU: a sum in the order that they count keeps them, and one row lost, or taken
twice, does not."""

import pytest
import torch

from norms_sums import depth, gradient_sums

SMS = 152


def kernel_order(terms, blocks, teams):
    """The sum over rows in 32 bits as the kernels add them: by team, by block, by warp of the second kernel, over warps."""
    t = terms.float()
    rows, width = t.shape
    by_team = torch.zeros(blocks * teams, width)
    for at in range(0, rows, blocks * teams):
        part = t[at:at + blocks * teams]
        by_team[:len(part)] += part
    by_block = torch.zeros(blocks, width)
    for k in range(teams):
        by_block += by_team.view(blocks, teams, width)[:, k]
    by_warp = torch.zeros(32, width)
    for at in range(0, blocks, 32):
        part = by_block[at:at + 32]
        by_warp[:len(part)] += part
    total = torch.zeros(width)
    for w in range(32):
        total += by_warp[w]
    return total


@pytest.mark.parametrize("rows, width, blocks, teams", [(257, 64, 5, 64), (20011, 64, 304, 64), (9000, 200, 304, 16),
                                                        (5000, 1024, 304, 4), (2500, 320, 152, 1), (40000, 40, 152, 1)])
def test_one_row_matters(rows, width, blocks, teams):
    g = torch.Generator().manual_seed(rows)
    x, d_y = torch.randn(rows, width, generator=g) + 0.3, torch.randn(rows, width, generator=g)
    n = (x.double() - x.double().mean(1, keepdim=True)) / (x.double().var(1, unbiased=False, keepdim=True) + 1e-5).sqrt()
    for name, (value, bound) in gradient_sums(x, d_y, SMS).items():
        terms = (d_y.double() * n if name == "d_gain" else d_y.double()).float()
        off = lambda t: (kernel_order(t, blocks, teams).double() - value).abs() > bound  # noqa: E731
        assert not off(terms).any(), name
        # Any column that is off shows it.  At 40000 rows, which the kernels' tests stay below, d_gain's bound is some 318 U of
        # 40000 * 0.64 and 140 U of 40000 * 0.8, 0.75 in all: a row's |d_y n| passes that in a quarter of its columns.
        for row in (0, rows // 2, rows - 1):
            lost = terms.clone()
            lost[row] = 0.0
            assert off(lost).any(), (name, row)
            twice = terms.clone()
            twice[row] *= 2
            assert off(twice).any(), (name, row)


def test_depth_of_few_rows():
    assert depth(1, SMS) == depth(256, SMS) == 256 and depth(257, SMS) == 130 + 152 // 8 + 1 + 32

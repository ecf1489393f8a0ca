"""The bound on dK of the few-rows backward tells the kernel's rule from others: mistakes planted in the 64-bit model."""

import pytest
import torch

import states_delta as sd


def worst(case, noted=None):
    """The largest ratio of error to bound over the items, of a model that notes states by `noted`."""
    rows, k_len, d = sd.CASES[case]
    g = torch.Generator().manual_seed(case)
    r = lambda n, scale=1.0: (scale * torch.randn(n, d, generator=g, dtype=torch.float64)).bfloat16()  # noqa: E731
    large, out = sd.large_weight(rows), 0.0
    for n in k_len * 4:
        q, k, v, d_o = (t.double() for t in (r(rows, 4.0), r(n), r(n), r(rows)))
        o = ((q @ k.T * d ** -0.5).softmax(-1) @ v).bfloat16().double()
        want, bound, got = sd.item(q, k, v, d_o, o, d ** -0.5, large, torch.bfloat16, noted)
        out = max(out, ((got.bfloat16().double() - want).abs() / bound).max().item())
    return out


@pytest.mark.parametrize("case", range(len(sd.CASES)))
def test_the_rule_is_within_the_bound_and_others_are_not(case):
    large = sd.large_weight(sd.CASES[case][0])
    assert worst(case) <= 1
    assert worst(case, lambda p: torch.zeros(p.shape[1], dtype=torch.bool)) > 1          # no state is noted
    assert worst(case, lambda p: p.amax(0) >= 2 * large) > 1                            # the limit is twice as high
    assert worst(case, lambda p: p[0] >= large) > 1 or p_rows(case) == 1                # only the first row is looked at


def p_rows(case):
    return sd.CASES[case][0]

"""Groups of experts whose sums of two choices fp32 cannot tell apart, because the terms are far larger than their sum
or than the scores in them, or cannot hold: the groups that stay are those of the real numbers."""

import pytest
import torch

from tests.test_gpu_route import _logits, check

pytestmark = pytest.mark.gpu

# experts, groups: a group in a part of a lane's experts, a whole lane's, several lanes', and across lanes
SIZES = [(16, 8), (32, 8), (64, 16), (96, 8), (256, 8), (250, 25), (512, 8), (1024, 32)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,groups", SIZES)
def test_sums_whose_terms_cancel(gpu, E, groups, score, dtype):
    """A group's two best have biases +B and -B, the others -3 B: its value is the sum of two scores, each
    rounded to |B| 2^-24 in fp32."""
    T, size = 2000, E // groups
    z = _logits(T, E, dtype, seed=E, std=0.01)
    for B in (16.0, 300.0, 1e4):
        bias = torch.full((groups, size), -3 * B)
        bias[:, 0], bias[:, -1] = -B, B
        for T0 in (T, 40):  # (few tokens take another shape of the kernel)
            check(gpu, z[:T0], min(6, E // 2), (B, T0), bias=bias.flatten(), score=score, groups=groups,
                  groups_kept=groups // 2, group_terms=2)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,groups", SIZES)
def test_sums_that_fp32_cannot_hold(gpu, E, groups, score):
    """Biases of the type's lowest and largest value: sums of two lie past its range, and such groups are there
    all the same."""
    size, kept = E // groups, groups // 2
    z = _logits(600, E, torch.float32, seed=E + 1)
    low = torch.finfo(torch.float32).min
    for value in (low, -2.0e38, -low):
        bias = torch.full((groups, size), value)
        bias[1], bias[-1] = 0.0, 0.01
        for T in (600, 40):
            for k in {min(12, 3 * size), 2}:
                if k <= kept * size:
                    check(gpu, z[:T], k, (value, T, k), bias=bias.flatten(), score=score, groups=groups,
                          groups_kept=kept, group_terms=2)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,groups", SIZES)
def test_far_away_groups_and_single_terms(gpu, E, groups, score):
    """Most groups at -1e30, fewer left than are kept; and groups by their best choice alone."""
    size, kept = E // groups, groups // 2
    z = _logits(600, E, torch.float32, seed=E + 2, std=0.01)
    bias = torch.full((groups, size), -1e30)
    bias[2], bias[3] = 50.0, 50.0
    for terms in (1, 2):
        check(gpu, z, min(6, 2 * size), terms, bias=bias.flatten(), score=score, groups=groups, groups_kept=kept,
              group_terms=terms)
        check(gpu, z, min(6, 2 * size), terms, bias=torch.full((E,), 1e4), score=score, groups=groups,
              groups_kept=kept, group_terms=terms)

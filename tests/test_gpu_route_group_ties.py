"""Groups whose sums of two choices are equal as real numbers, with the terms of one rounded otherwise than those of
another: the lowest groups stay."""

import pytest
import torch

from fp8_fine_grained_amd import experts as ex

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("k", [4, 20])  # (more than 15: a kernel of its own)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("groups,size", [(8, 4), (16, 16), (5, 7), (64, 4)])
def test_biases_the_other_way_round(gpu, groups, size, score, dtype, k):
    """Every group has the same two good logits; every other one has their biases the other way round."""
    kept = min(groups // 2, max(3, groups // 3))
    k = min(k, kept * size)
    T = 1000
    g = torch.Generator().manual_seed(groups)
    z = torch.full((T, groups, size), -9.0)
    z[:, :, 1:3] = torch.randn((T, 1, 2), generator=g) * 0.5
    for b in (torch.tensor([0.3, 0.1]), torch.tensor([1.7, 100.3]), torch.tensor([0.05, 0.02])):
        bias = torch.zeros((groups, size))
        bias[0::2, 1:3], bias[1::2, 1:3] = b, b.flip(0)
        for rows in (T, 30):
            experts, _ = ex.route_experts(z.view(T, -1)[:rows].to(dtype).to(gpu), k, bias=bias.flatten().to(gpu),
                                          score=score, groups=groups, groups_kept=kept)
            at = experts.cpu() // size
            assert torch.all((at >= 0) & (at < kept)), (b, rows, int((at >= kept).any(1).sum()))

"""More rows than one launch can count (2^32 work-items along x)."""

import pytest
import torch

from fp8_fine_grained_amd import layer
from tests.gpu_util import say

pytestmark = pytest.mark.gpu


def test_norm_of_more_rows_than_a_launch_holds(gpu):
    """128-wide rows, a wavefront each: the second launch starts at row 2^26 - 4.  Every
    row repeats one of 4096, so each output has to repeat those rows' own."""
    H, P = 128, 4096
    M = (1 << 26) + 4096
    say(f"norm {M}x{H}")
    g = torch.Generator(device="cuda").manual_seed(0)
    few, res = (torch.randn((P, H), generator=g, device=gpu).to(torch.bfloat16) for _ in range(2))
    w = torch.rand(H, generator=g, device=gpu) + 0.5
    y1 = torch.empty_like(few)
    want = (*layer.fp8_add_rmsnorm_quant_1x128(few, w, residual=res, y=y1), y1)
    x, r = few.repeat(M // P, 1), res.repeat(M // P, 1)
    y = torch.full_like(x, float("nan"))
    got = (*layer.fp8_add_rmsnorm_quant_1x128(x, w, residual=r, y=y), y)
    del x, r
    for name, a, b in zip(("h", "codes", "scales", "rstd", "y"), got, want):
        a = a.view(M // P, *b.shape)
        for i in range(0, M // P, 2048):
            part = a[i:i + 2048]
            assert torch.equal(part, b.expand_as(part)), f"{name}, rows from {i * P}"

"""The sigmoid routing gradient of confident experts: 1 - s is exp(-z) there, far below the rounding of s."""

import pytest
import torch

from fp8_fine_grained_amd import experts as ex
from tests import experts_reference as ref
from tests.layer_reference import U, UB

pytestmark = pytest.mark.gpu


def gradient(dw, at, z, renormalise, scale, ds):
    """(dz, the magnitudes that its roundings are relative to) in 64 bits, with 1 - s as sigmoid(-z)."""
    z, g = z.double(), dw.double() * scale
    s = torch.sigmoid(z)
    if renormalise:
        p = ref.shares(z, at, torch.ones_like(at, dtype=torch.bool), "sigmoid")
        mean = (g * p).sum(dim=1, keepdim=True)
        t, ta = p * (g - mean), p * (g.abs() + (g * p).abs().sum(dim=1, keepdim=True))
    else:
        q = s.gather(1, at)
        t, ta = q * g, (q * g).abs()
    d, da = torch.zeros_like(z).scatter_add_(1, at, t), torch.zeros_like(z).scatter_add_(1, at, ta)
    if ds is not None:
        d, da = d + ds.double() * s, da + (ds.double() * s).abs()
    return d * torch.sigmoid(-z), da * torch.sigmoid(-z)


@pytest.mark.parametrize("renormalise", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,k", [(60, 4), (128, 8), (256, 8), (512, 8), (1000, 32)])
def test_gradient_of_large_logits(gpu, E, k, dtype, renormalise):
    T = 64
    g = torch.Generator().manual_seed(E)
    z = (torch.rand((T, E), generator=g) * 35 + 5).to(dtype)
    z[::4] -= 20                                       # from -15 to 20
    experts = torch.rand((T, E), generator=g).argsort(dim=1)[:, :k]
    dw, ds = torch.randn((T, k), generator=g), torch.randn((T, E), generator=g)
    for d in (None, ds):
        got = ex.route_experts_backward(dw.to(gpu), experts.int().to(gpu), z.to(gpu), score="sigmoid",
                                        renormalise=renormalise, scale=2.5, dscores=None if d is None else d.to(gpu))
        want, size = gradient(dw, experts, z, renormalise, 2.5, d)
        # scores of chosen experts, of their sum, and of the factor (6 roundings each); sums over up to 32 places and
        # the products (40); the rounding to the output's type
        tol = (3 * 6 + 40) * U * size + (UB if dtype == torch.bfloat16 else U) * want.abs()
        off = (got.cpu().double() - want).abs()
        assert torch.all(off <= tol), float((off / tol).nan_to_num(0.0).max())


def test_gradient_at_the_ends(gpu):
    """Infinite logits and those past the exponential's range."""
    z = torch.tensor([[float("inf"), 200.0, 88.0, 30.0, -30.0, -88.0, -200.0, -float("inf")]])
    at = torch.arange(8)[None]
    dw = torch.full((1, 8), 3.0)
    got = ex.route_experts_backward(dw.to(gpu), at.int().to(gpu), z.to(gpu), score="sigmoid", renormalise=False)
    want = 3.0 * torch.sigmoid(z.double()) * torch.sigmoid(-z.double())
    # (scores below the normal range may be lost)
    assert torch.all((got.cpu().double() - want).abs() <= 58 * U * want + 3 * 2.0 ** -126)

"""The oracle of the layer operators' quantised outputs sees codes that are not numbers."""

import pytest
import torch

from tests.layer_reference import E4M3_MAX, check_quant


def _quantised(pow2):
    """Values [4, 256], their codes and their scales, all exact: powers of two."""
    ref = torch.exp2(torch.arange(4 * 256).remainder(5).double()).view(4, 256)
    ref[:, ::3] *= -1
    s = torch.full((4, 2), 16 / (256.0 if pow2 else E4M3_MAX))
    v = ref.view(4, 2, 128) / s[:, :, None].double()
    return ref, v.float().to(torch.float8_e4m3fn).view(torch.uint8).view(4, 256), s


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("code", [0x7F, 0xFF])
def test_codes_that_are_not_numbers_are_rejected(pow2, code):
    ref, q, s = _quantised(pow2)
    check_quant(q, s, ref, 0.0, pow2)
    for at in ((1, 7), (2, slice(None)), (3, slice(128, 256)), (slice(None), slice(None))):
        bad = q.clone()
        bad[at] = code
        with pytest.raises(AssertionError, match="codes off"):
            check_quant(bad, s, ref, 0.0, pow2)


@pytest.mark.parametrize("pow2", [False, True])
def test_scales_that_are_not_numbers_are_rejected(pow2):
    ref, q, s = _quantised(pow2)
    s[2, 1] = float("nan")
    with pytest.raises(AssertionError):
        check_quant(q, s, ref, 0.0, pow2)

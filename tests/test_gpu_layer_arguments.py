"""Arguments that the layer operators' Python entry points refuse before anything is launched."""

import pytest
import torch

from fp8_fine_grained_amd import layer
from tests.test_gpu_gated import _operands

pytestmark = pytest.mark.gpu


def test_the_dense_gated_product_takes_one_weight(gpu):
    """A stack of experts' weights is not silently taken for its first one."""
    qa, sa, qw, sw = _operands(gpu, 4, 128, 256, False, G=2)
    for call in (layer.fp8_block_gated_gemm, layer.fp8_block_gated_gemm_quant):
        with pytest.raises(ValueError):
            call(qa, sa, qw, sw)
        with pytest.raises(ValueError):
            call(qa, sa, qw[:1], sw[:1])
        call(qa, sa, qw[0], sw[0])

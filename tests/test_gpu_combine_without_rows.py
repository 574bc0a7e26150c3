"""The combination's gradient on a GPU that holds none of the rows, or of rows without columns."""

import pytest
import torch

from fp8_fine_grained_amd import binding
from fp8_fine_grained_amd import experts as ex

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_no_rows(gpu, dtype):
    dy = torch.ones((3, 128), dtype=dtype, device=gpu)
    gone = torch.tensor([[-1, 0], [5, -1], [-1, -1]], dtype=torch.int32, device=gpu)
    w = torch.ones((3, 2), device=gpu)
    for weights in (w, None):
        d, dw = ex.combine_experts_backward(dy, gone, weights, R=0)
        assert d.shape == (0, 128) and dw is None
        d, dw = ex.combine_experts_backward(dy, gone, weights, rows=dy[:0], need_dweights=False)
        assert d.shape == (0, 128) and dw is None
        d, dw = ex.combine_experts_backward(dy, gone, weights, rows=dy[:0], need_drows=False)
        assert d is None and torch.all(dw == 0)
        for pow2 in (False, True):
            q, s, dw = ex.combine_experts_backward_quant(dy, gone, weights, R=0, pow2=pow2)
            assert q.shape == (0, 128) and s.shape == (0, 1) and dw is None
            q, s, dw = ex.combine_experts_backward_quant(dy, gone, weights, rows=dy[:0], need_dweights=False)
            assert q.shape == (0, 128) and s.shape == (0, 1) and dw is None
            q, s, dw = ex.combine_experts_backward_quant(dy, gone, weights, rows=dy[:0], pow2=pow2)
            assert q.shape == (0, 128) and torch.all(dw == 0)


def test_no_columns(gpu):
    dy = torch.ones((3, 0), device=gpu)
    at = torch.arange(6, dtype=torch.int32, device=gpu).view(3, 2)
    d, dw = ex.combine_experts_backward(dy, at, R=6)
    assert d.shape == (6, 0) and dw is None
    d, dw = ex.combine_experts_backward(dy, at, rows=torch.ones((6, 0), device=gpu))
    assert d.shape == (6, 0) and torch.all(dw == 0)
    q, s, dw = ex.combine_experts_backward_quant(dy, at, R=6)
    assert q.shape == (6, 0) and s.shape == (6, 0) and dw is None


def test_an_output_has_to_be_asked_for(gpu):
    dy = torch.ones((3, 128), device=gpu)
    at = torch.arange(6, dtype=torch.int32, device=gpu).view(3, 2)
    with pytest.raises(binding.Fp8fgError):
        ex.combine_experts_backward(dy, at, need_drows=False)

"""Products with 4-bit weights over the longest segments."""

import pytest
import torch

from fp8_fine_grained_amd import experts as ex
from tests import experts_reference as ref
from tests.gpu_util import say
from tests.test_gpu_fp4 import exact_operands, on

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("codes", [False, True])
def test_a_segment_of_every_row_that_can_be_counted(gpu, codes):
    """2^31 - 1 rows of 1009 tokens, all of them one expert's: each has to repeat its token's own product."""
    M, T = 2 ** 31 - 1, 1009
    say(f"{M} rows, codes {codes}")
    x, sx, w, sw = exact_operands(T, 1, 128, codes, G=2)
    want = (ref.x_values(x, sx) @ ref.fp4_values(w[1], sw[1]).t()).float().to(torch.bfloat16).to(gpu)
    xs, sxs, ws, sws = on(gpu, x, sx, w, sw)
    index = torch.arange(M, dtype=torch.int32, device=gpu)
    index.remainder_(T)
    offsets = torch.tensor([0, 0, M], dtype=torch.int32, device=gpu)
    y = torch.full((M, 1), 7.0, dtype=torch.bfloat16, device=gpu)
    ex.fp4_grouped_gemm(xs, offsets, ws, sws, sx=sxs, row_index=index, y=y)
    del index
    step = T << 15
    tokens = want.repeat(1 << 15, 1)
    for r in range(0, M, step):
        part = y[r:r + step]
        assert torch.equal(part, tokens[:part.shape[0]]), r

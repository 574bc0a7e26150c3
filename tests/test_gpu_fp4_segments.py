"""Products with 4-bit weights over expert segments in every workgroup shape (tests/test_fp4_segment_shapes.py): ragged
segments, one of them empty, rows read by index or as they come."""

import pytest
import torch

from fp8_fine_grained_amd import experts as ex
from tests import experts_reference as ref
from tests.layer_reference import U, silu
from tests.test_gpu_fp4 import exact_operands, on

pytestmark = pytest.mark.gpu

EXPERTS = 4
# Rows and columns (of the plain product; gated: half as many) that take every workgroup shape in turn.
SEGMENTED = [(1, 40), (2, 2090), (2, 4140), (100, 70), (4, 1066), (4, 2090), (21, 550), (21, 1574), (50, 1060),
             (21, 2090), (21, 3110), (50, 1574), (50, 2090)]


def _counts(M):
    """Rows of each expert; the second has none."""
    return [M // 3, 0, M - M // 3 - M // 4, M // 4]


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("M,N", SEGMENTED)
def test_every_workgroup_shape_over_segments(gpu, M, N, codes, gated):
    """K: fewer 128s than wavefronts share it, an odd number of them, more than the rings hold."""
    offsets = torch.tensor([0, *torch.tensor(_counts(M)).cumsum(0).tolist()], dtype=torch.int32)
    T = M // 2 + 1
    rows = torch.randint(0, T, (M,), generator=torch.Generator().manual_seed(M)).int()
    call = ex.fp4_grouped_gated_gemm if gated else ex.fp4_grouped_gemm
    for K in (128, 384, 2176):
        for index in (rows, None):
            x, sx, w, sw = exact_operands(M if index is None else T, N, K, codes, seed=K + M, G=EXPERTS)
            sw -= 4 if gated else 0
            v = ref.x_values(x, sx)
            v = v if index is None else v[index.long()]
            want = torch.cat([v[offsets[e]:offsets[e + 1]] @ ref.fp4_values(w[e], sw[e]).t() for e in range(EXPERTS)])
            xs, sxs, ws, sws, o, i = on(gpu, x, sx, w, sw, offsets, index)
            room = torch.full((M + 8, N // 2 if gated else N), 7.0, device=gpu)
            given = dict(h=room[4:M + 4]) if gated else dict(y=room[4:M + 4])
            call(xs, o, ws, sws, sx=sxs, row_index=i, **given)
            assert torch.all(room[:4] == 7) and torch.all(room[M + 4:] == 7)
            got = room[4:M + 4].cpu().double()
            if gated:
                h = silu(want[:, :N // 2]) * want[:, N // 2:]
                assert torch.all((got - h).abs() <= 10 * U * h.abs() + 2.0 ** -100), K
            else:
                assert torch.equal(got, want), K

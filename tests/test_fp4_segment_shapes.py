"""The GPU tests take every workgroup shape of the products with 4-bit weights over expert segments, in every form."""

import pytest

from tests.test_fp4_shapes import choose  # noqa: F401  (a fixture)
from tests.test_gpu_fp4_segments import EXPERTS, SEGMENTED


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("codes", [False, True])
def test_every_shape_over_segments(choose, codes, gated):  # noqa: F811
    count, shapes = choose(*[(M, N // 2 if gated else N, EXPERTS, True, gated, codes) for M, N in SEGMENTED])
    assert sorted(set(shapes)) == list(range(count)), shapes

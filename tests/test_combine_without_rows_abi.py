"""The combination's gradient of no rows, or of rows without columns, asked for without dweights: nothing to do, and the
absent rows need no address (no call here launches a kernel)."""

import pytest

from fp8_fine_grained_amd import binding as fp8
from fp8_fine_grained_amd import experts as ex
from tests.test_experts_abi import COMBINE_GRAD, COMBINE_QUANT, GOOD, NULL, ODDER, _caller


@pytest.mark.parametrize("empty", [dict(R=0), dict(H=0), dict(R=0, H=0)])
def test_nothing_to_do(empty):
    L = ex.lib()
    f = _caller(L.fp8fg_combine_experts_backward, COMBINE_GRAD)
    for rows in (NULL, GOOD):
        for drows in (NULL, GOOD, ODDER):
            assert f(dw=NULL, rows=rows, drows=drows, **empty) == fp8.OK, (rows, drows)
    assert f(dw=NULL, drows=NULL, dt=7, **empty) == fp8.ERR_INVALID_ARG
    assert f(dw=NULL, drows=NULL, positions=NULL, **empty) == fp8.ERR_INVALID_ARG
    f = _caller(L.fp8fg_combine_experts_backward_quant, COMBINE_QUANT)
    for pow2 in (0, 1):
        assert f(dw=NULL, rows=NULL, drows=NULL, scales=NULL, pow2=pow2, **empty) == fp8.OK

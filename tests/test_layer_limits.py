"""Sizes whose launches HIP could not count (2^32 work-items along x): refused on the host, before
any HIP call, at the limits that include/fp8fg_layer.h states."""

import pytest

from fp8_fine_grained_amd import binding as fp8
from tests.test_layer_abi import GATED, GOOD, NULL, PLAIN_OUT, QUANT_OUT, SEGMENTS, L, _caller  # noqa: F401

TILES = 8388600


@pytest.mark.parametrize("fn,ok", [("fp8_block_gated_gemm", {**GATED, **PLAIN_OUT}),
                                   ("fp8_block_gated_gemm_quant", {**GATED, **QUANT_OUT})])
def test_gated_tiles(L, fn, ok):  # noqa: F811
    f = _caller(getattr(L, fn), ok)
    assert f(M=(TILES + 1) * 128) == fp8.ERR_UNSUPPORTED
    assert f(M=TILES * 128 + 1) == fp8.ERR_UNSUPPORTED
    assert f(M=1, I=(TILES + 1) * 128) == fp8.ERR_UNSUPPORTED
    assert f(M=1 << 20, I=1 << 18) == fp8.ERR_UNSUPPORTED


@pytest.mark.parametrize("fn,ok", [("fp8_block_grouped_gated_gemm", {**SEGMENTS, **PLAIN_OUT}),
                                   ("fp8_block_grouped_gated_gemm_quant", {**SEGMENTS, **QUANT_OUT})])
def test_gated_tiles_over_experts(L, fn, ok):  # noqa: F811
    f = _caller(getattr(L, fn), ok)
    assert f(M=(TILES - 3) * 128) == fp8.ERR_UNSUPPORTED  # (4 experts)
    assert f(G=TILES + 1) == fp8.ERR_UNSUPPORTED


def test_gated_backward(L):  # noqa: F811
    f = _caller(L.fp8_gated_backward_quant, dict(dh=GOOD, gu=GOOD, dt=fp8.BF16, M=128, I=128, ld=1 << 31, pow2=0,
                                                 q=GOOD, s=GOOD, qt=GOOD, st=GOOD, qht=GOOD, sht=GOOD, stream=NULL))
    rows = dict(qt=NULL, st=NULL, qht=NULL, sht=NULL)
    assert f(M=(1 << 28) - 15, **rows) == fp8.ERR_UNSUPPORTED
    assert f(M=1 << 20, I=1 << 15, **rows) == fp8.ERR_UNSUPPORTED
    assert f(dt=fp8.F32, M=(1 << 20) + 128, I=1 << 17) == fp8.ERR_UNSUPPORTED
    assert f(dt=fp8.F32, M=TILES * 128 + 128) == fp8.ERR_UNSUPPORTED
    # within them the next check is reached
    assert f(M=(1 << 28) - 16, dh=NULL, **rows) == fp8.ERR_INVALID_ARG
    assert f(dt=fp8.F32, M=TILES * 128, dh=NULL) == fp8.ERR_INVALID_ARG
    assert f(dt=fp8.BF16, M=TILES * 128 + 128, dh=NULL) == fp8.ERR_INVALID_ARG

"""include/fp8fg_experts.h: every declared function is exported and bound, and invalid arguments are refused
on the host (no call here launches a kernel)."""

import ctypes
import re

import pytest

from fp8_fine_grained_amd import binding as fp8
from fp8_fine_grained_amd import experts as ex

BAD = ctypes.c_void_p(0x1008)   # 8-byte aligned, not 16: never dereferenced
GOOD = ctypes.c_void_p(0x10000)  # aligned stand-in: only used where validation fails first
ODD = ctypes.c_void_p(0x10002)
ODDER = ctypes.c_void_p(0x10001)
NULL = ctypes.c_void_p(0)
BIG = 1 << 31


@pytest.fixture(scope="module")
def L():
    return ex.lib()


def _caller(f, ok):
    def call(**kw):
        assert set(kw) <= set(ok)
        return f(*[kw.get(k, v) for k, v in ok.items()])
    return call


def test_exports_and_binds_every_declared_function(L):
    names = set(re.findall(r"^(?:int|int64_t)\s+(\w+)\s*\(", open(ex.HEADER).read(), flags=re.M))
    assert names == set(ex._SIGS)
    for n in names:
        assert hasattr(L, n), n


ROUTE = dict(z=GOOD, dt=fp8.F32, T=4, E=64, ld=64, bias=GOOD, mask=GOOD, score=1, groups=8, kept=4, terms=2, k=8,
             renorm=1, scale=1.0, experts=GOOD, weights=GOOD, scores=GOOD, stream=NULL)
ROUTE_GRAD = dict(dw=GOOD, experts=GOOD, z=GOOD, dt=fp8.F32, T=4, E=64, ld=64, score=1, k=8, renorm=1, scale=1.0,
                  ds=GOOD, dz=GOOD, stream=NULL)


def test_routing_validation(L):
    for f, bad in ((_caller(L.fp8fg_route_experts, ROUTE), "experts weights"),
                   (_caller(L.fp8fg_route_experts_backward, ROUTE_GRAD), "dw experts dz")):
        for k, v in (("dt", 2), ("T", -1), ("E", -1), ("k", -1), ("score", 2), ("score", -1), ("renorm", 2),
                     ("scale", float("nan")), ("scale", float("inf")), ("z", NULL), ("ld", 63)):
            assert f(**{k: v}) == fp8.ERR_INVALID_ARG, k
        for kw in (dict(E=1032, ld=1032), dict(k=33), dict(E=0), dict(k=0), dict(T=BIG), dict(ld=1 << 60)):
            assert f(**kw) == fp8.ERR_UNSUPPORTED, kw
        for k in bad.split():
            assert f(**{k: NULL}) == fp8.ERR_INVALID_ARG, k
            assert f(**{k: ODD}) == fp8.ERR_MISALIGNED, k
        assert f(z=ODD) == fp8.ERR_MISALIGNED
        assert f(z=ODDER, dt=fp8.BF16) == fp8.ERR_MISALIGNED
        assert f(T=0, z=NULL, experts=NULL) == fp8.OK
    f = _caller(L.fp8fg_route_experts, ROUTE)
    for kw in (dict(groups=0), dict(kept=0), dict(kept=9), dict(terms=0), dict(terms=3)):
        assert f(**kw) == fp8.ERR_INVALID_ARG, kw
    for kw in (dict(groups=7), dict(kept=1, k=9), dict(E=128, ld=128, groups=128, kept=8),
               dict(groups=64, kept=32, terms=2)):
        assert f(**kw) == fp8.ERR_UNSUPPORTED, kw
    assert f(bias=ODD) == fp8.ERR_MISALIGNED and f(scores=ODD) == fp8.ERR_MISALIGNED
    f = _caller(L.fp8fg_route_experts_backward, ROUTE_GRAD)
    assert f(k=65) == fp8.ERR_UNSUPPORTED and f(E=7, ld=7) == fp8.ERR_UNSUPPORTED  # k > E
    assert f(ds=ODD) == fp8.ERR_MISALIGNED


def test_segments_validation(L):
    f = _caller(L.fp8fg_expert_segments, dict(experts=GOOD, T=4096, k=8, first=0, G=16, offsets=GOOD, rows=GOOD,
                                              positions=GOOD, ws=GOOD, bytes=1 << 30, stream=NULL))
    for k in ("T", "k", "first", "G"):
        assert f(**{k: -1}) == fp8.ERR_INVALID_ARG
    for kw in (dict(G=0), dict(G=1025), dict(first=BIG - 16), dict(T=1 << 28)):
        assert f(**kw) == fp8.ERR_UNSUPPORTED, kw
    for k in ("experts", "offsets", "rows", "positions"):
        assert f(**{k: NULL}) == fp8.ERR_INVALID_ARG, k
        assert f(**{k: ODD}) == fp8.ERR_MISALIGNED, k
    need = L.fp8fg_expert_segments_workspace(4096, 8, 16)
    assert need > 0
    assert f(ws=NULL) == fp8.ERR_INVALID_ARG and f(bytes=need - 1) == fp8.ERR_INVALID_ARG
    assert f(ws=ODD) == fp8.ERR_MISALIGNED
    for T, k, G in ((0, 8, 16), (8, 0, 16), (-1, 8, 16), (8, 8, 0), (8, 8, 2000), (BIG, 8, 4)):
        assert L.fp8fg_expert_segments_workspace(T, k, G) == 0


COMBINE = dict(rows=GOOD, dt=fp8.BF16, R=16, H=256, ld=256, positions=GOOD, w=GOOD, T=4, k=4, base=GOOD, ldb=256,
               y=GOOD, stream=NULL)
COMBINE_GRAD = dict(dy=GOOD, rows=GOOD, dt=fp8.BF16, R=16, H=256, ldy=256, ld=256, positions=GOOD, w=GOOD, T=4, k=4,
                    drows=GOOD, dw=GOOD, stream=NULL)
COMBINE_QUANT = dict(dy=GOOD, rows=GOOD, dt=fp8.BF16, R=16, H=256, ldy=256, ld=256, positions=GOOD, w=GOOD, T=4, k=4,
                     pow2=0, drows=GOOD, scales=GOOD, dw=GOOD, stream=NULL)


@pytest.mark.parametrize("name,ok,wide,given", [
    ("fp8fg_combine_experts", COMBINE, "rows base y", "rows positions y"),
    ("fp8fg_combine_experts_backward", COMBINE_GRAD, "dy rows drows", "dy rows positions"),
    ("fp8fg_combine_experts_backward_quant", COMBINE_QUANT, "dy rows drows", "dy rows positions drows scales")])
def test_combine_validation(L, name, ok, wide, given):
    f = _caller(getattr(L, name), ok)
    for k in ("R", "H", "T", "k"):
        assert f(**{k: -1}) == fp8.ERR_INVALID_ARG, k
        assert f(**{k: BIG}) == fp8.ERR_UNSUPPORTED, k
    assert f(dt=3) == fp8.ERR_INVALID_ARG
    assert f(H=252) == fp8.ERR_UNSUPPORTED and f(k=33) == fp8.ERR_UNSUPPORTED
    for k in given.split():
        assert f(**{k: NULL}) == fp8.ERR_INVALID_ARG, k
    for k in wide.split():
        assert f(**{k: BAD}) == fp8.ERR_MISALIGNED, k
    for k in ("ld", "ldb", "ldy"):
        if k in ok:
            assert f(**{k: 255}) == fp8.ERR_INVALID_ARG
            assert f(**{k: 260}) == fp8.ERR_MISALIGNED
            assert f(**{k: 1 << 60}) == fp8.ERR_UNSUPPORTED
    for k in ("positions", "w", "dw", "scales"):
        if k in ok:
            assert f(**{k: ODD}) == fp8.ERR_MISALIGNED, k
    if "dw" in ok:
        assert f(T=0) == fp8.OK and f(k=0) == fp8.OK
    else:
        assert f(T=0) == fp8.OK and f(H=0) == fp8.OK
    if name.endswith("quant"):
        assert f(H=200) == fp8.ERR_UNSUPPORTED and f(pow2=2) == fp8.ERR_INVALID_ARG
    if name.endswith("backward"):
        assert f(drows=NULL, dw=NULL) == fp8.ERR_INVALID_ARG


def test_fp4_quant_validation(L):
    f = _caller(L.fp4_quant_weight_1x32, dict(w=GOOD, dt=fp8.BF16, N=4, K=256, ld=256, q=GOOD, s=GOOD, stream=NULL))
    assert f(dt=2) == f(N=-1) == f(K=-1) == f(ld=255) == fp8.ERR_INVALID_ARG
    assert f(K=192) == f(N=1 << 27) == f(N=1 << 62) == f(ld=1 << 60) == fp8.ERR_UNSUPPORTED
    for k in ("w", "q", "s"):
        assert f(**{k: NULL}) == fp8.ERR_INVALID_ARG
    assert f(w=BAD) == f(q=BAD) == f(s=ODD) == f(ld=260) == fp8.ERR_MISALIGNED
    assert f(N=0, w=NULL) == f(K=0) == fp8.OK


DENSE = dict(x=GOOD, sx=GOOD, w=GOOD, sw=GOOD, y=GOOD, dt=fp8.BF16, M=4, N=96, K=256, stream=NULL)
GROUPED = dict(x=GOOD, sx=GOOD, T=4, rows=GOOD, offsets=GOOD, G=3, w=GOOD, sw=GOOD, y=GOOD, dt=fp8.BF16, M=4, N=96,
               K=256, stream=NULL)


@pytest.mark.parametrize("name", ["fp4_gemm", "fp4_gated_gemm", "fp4_grouped_gemm", "fp4_grouped_gated_gemm"])
def test_fp4_validation(L, name):
    grouped = "grouped" in name
    f = _caller(getattr(L, name), GROUPED if grouped else DENSE)
    assert f(dt=2) == fp8.ERR_INVALID_ARG
    for k in ("M", "N", "K") + (("T", "G") if grouped else ()):
        assert f(**{k: -1}) == fp8.ERR_INVALID_ARG, k
        assert f(**{k: BIG}) == fp8.ERR_UNSUPPORTED, k
    assert f(K=0) == f(K=192) == f(K=1 << 24) == fp8.ERR_UNSUPPORTED
    for k in ("x", "w", "sw", "y") + (("offsets",) if grouped else ()):
        assert f(**{k: NULL}) == fp8.ERR_INVALID_ARG, k
    assert f(x=BAD) == f(w=BAD) == f(sx=ODD) == f(sw=ODD) == f(y=ODDER) == fp8.ERR_MISALIGNED
    assert f(y=ODD, dt=fp8.F32) == fp8.ERR_MISALIGNED
    assert f(M=BIG - 1, N=BIG - 1, **(dict(T=BIG - 1) if grouped else {})) == fp8.ERR_UNSUPPORTED  # work-items
    assert f(M=0) == f(N=0) == fp8.OK
    if grouped:
        assert f(T=0) == f(rows=NULL, T=5) == fp8.ERR_INVALID_ARG
        assert f(offsets=ODD) == f(rows=ODD) == fp8.ERR_MISALIGNED
        assert f(G=BIG - 1, K=(1 << 24) - 128, N=BIG - 1) == fp8.ERR_UNSUPPORTED
        assert f(G=0) == fp8.OK

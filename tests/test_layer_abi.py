"""include/fp8fg_layer.h: every declared function is exported and bound, and
invalid arguments are refused on the host (no call here launches a kernel)."""

import ctypes
import re

import pytest

from fp8_fine_grained_amd import binding as fp8
from fp8_fine_grained_amd import layer

BAD = ctypes.c_void_p(0x1008)   # 8-byte aligned, not 16: never dereferenced
GOOD = ctypes.c_void_p(0x10000)  # aligned stand-in: only used where validation fails first
ODD = ctypes.c_void_p(0x10002)
NULL = ctypes.c_void_p(0)


@pytest.fixture(scope="module")
def L():
    return layer.lib()


def test_exports_and_binds_every_declared_function(L):
    names = set(re.findall(r"^(?:int|int64_t)\s+(\w+)\s*\(", open(layer.HEADER).read(), flags=re.M))
    assert names == set(layer._SIGS)
    for n in names:
        assert hasattr(L, n), n


def _caller(f, ok):
    def call(**kw):
        assert set(kw) <= set(ok)
        return f(*[kw.get(k, v) for k, v in ok.items()])
    return call


def test_norm_validation(L):
    f = _caller(L.fp8_add_rmsnorm_quant_1x128, dict(
        x=GOOD, r=GOOD, dt=fp8.BF16, M=4, H=256, ldx=256, ldr=256, w=GOOD, wdt=fp8.F32, eps=1e-6, pow2=0, h=GOOD,
        y=NULL, q=GOOD, s=GOOD, rstd=GOOD, stream=NULL))
    assert f(dt=7) == fp8.ERR_INVALID_ARG
    assert f(wdt=7) == fp8.ERR_INVALID_ARG
    assert f(M=-1) == fp8.ERR_INVALID_ARG
    assert f(H=200, ldx=200, ldr=200) == fp8.ERR_UNSUPPORTED
    assert f(H=32768 + 128, ldx=1 << 16, ldr=1 << 16) == fp8.ERR_UNSUPPORTED
    assert f(M=1 << 31) == fp8.ERR_UNSUPPORTED
    assert f(eps=-1.0) == fp8.ERR_INVALID_ARG
    assert f(eps=float("nan")) == fp8.ERR_INVALID_ARG
    assert f(pow2=2) == fp8.ERR_INVALID_ARG
    assert f(ldx=255) == fp8.ERR_INVALID_ARG
    assert f(ldr=128) == fp8.ERR_INVALID_ARG
    for k in ("x", "w", "q", "s"):
        assert f(**{k: NULL}) == fp8.ERR_INVALID_ARG
    for k in ("x", "r", "w", "h", "y", "q"):
        assert f(**{k: BAD}) == fp8.ERR_MISALIGNED
    assert f(s=ODD) == fp8.ERR_MISALIGNED
    assert f(rstd=ODD) == fp8.ERR_MISALIGNED
    assert f(ldx=260) == fp8.ERR_MISALIGNED  # 520 bytes
    assert f(M=0, x=NULL, q=NULL, s=NULL) == fp8.OK


def test_norm_backward_validation(L):
    need = L.fp8_rmsnorm_backward_workspace(4, 256)
    assert need > 0 and need % 1024 == 0
    assert L.fp8_rmsnorm_backward_workspace(0, 256) == 0
    assert L.fp8_rmsnorm_backward_workspace(-1, 256) == 0
    f = _caller(L.fp8_rmsnorm_backward, dict(
        dy=GOOD, h=GOOD, dh=GOOD, dt=fp8.BF16, M=4, H=256, ldy=256, ldh=256, lddh=256, rstd=GOOD, w=GOOD, wdt=fp8.F32,
        dx=GOOD, dw=GOOD, ws=GOOD, bytes=need, stream=NULL))
    assert f(dt=2) == fp8.ERR_INVALID_ARG
    assert f(H=192, ldy=192, ldh=192, lddh=192) == fp8.ERR_UNSUPPORTED
    assert f(bytes=need - 1) == fp8.ERR_INVALID_ARG
    assert f(ws=NULL) == fp8.ERR_INVALID_ARG
    assert f(ws=BAD) == fp8.ERR_MISALIGNED
    assert f(dw=BAD) == fp8.ERR_MISALIGNED
    for k in ("dy", "h", "rstd", "w", "dx"):
        assert f(**{k: NULL}) == fp8.ERR_INVALID_ARG
    for k in ("dy", "h", "dh", "w", "dx"):
        assert f(**{k: BAD}) == fp8.ERR_MISALIGNED
    for k in ("ldy", "ldh", "lddh"):
        assert f(**{k: 128}) == fp8.ERR_INVALID_ARG
    assert f(M=0, dw=NULL, dy=NULL) == fp8.OK  # nothing to write


GATED = dict(a=GOOD, sa=GOOD, w=GOOD, sw=GOOD, accum=fp8.ACCUM_FP8_MFMA)
SEGMENTS = dict(a=GOOD, sa=GOOD, T=32, idx=GOOD, off=GOOD, G=4, w=GOOD, sw=GOOD, accum=fp8.ACCUM_FP8_MFMA)
PLAIN_OUT = dict(h=GOOD, dt=fp8.BF16, gu=GOOD, M=4, I=128, K=256, stream=NULL)
QUANT_OUT = dict(pow2=0, h=GOOD, s=GOOD, gu=GOOD, ws=GOOD, bytes=1 << 20, M=4, I=128, K=256, stream=NULL)


@pytest.mark.parametrize("fn,ok", [("fp8_block_gated_gemm", {**GATED, **PLAIN_OUT}),
                                   ("fp8_block_gated_gemm_quant", {**GATED, **QUANT_OUT}),
                                   ("fp8_block_grouped_gated_gemm", {**SEGMENTS, **PLAIN_OUT}),
                                   ("fp8_block_grouped_gated_gemm_quant", {**SEGMENTS, **QUANT_OUT})])
def test_gated_validation(L, fn, ok):
    f = _caller(getattr(L, fn), ok)
    assert f(accum=9) == fp8.ERR_INVALID_ARG
    assert f(M=-1) == fp8.ERR_INVALID_ARG
    assert f(I=-128) == fp8.ERR_INVALID_ARG
    assert f(I=64) == fp8.ERR_UNSUPPORTED
    assert f(K=0) == fp8.ERR_UNSUPPORTED
    assert f(K=200) == fp8.ERR_UNSUPPORTED
    assert f(K=1 << 24) == fp8.ERR_UNSUPPORTED
    assert f(M=1 << 31) == fp8.ERR_UNSUPPORTED
    assert f(I=1 << 30) == fp8.ERR_UNSUPPORTED
    for k in ("a", "sa", "w", "sw", "h"):
        assert f(**{k: NULL}) == fp8.ERR_INVALID_ARG
    for k in ("a", "w", "h", "gu"):
        assert f(**{k: BAD}) == fp8.ERR_MISALIGNED
    assert f(sa=ctypes.c_void_p(0x10001)) == fp8.ERR_MISALIGNED
    assert f(M=0, a=NULL) == fp8.OK
    assert f(I=0, a=NULL) == fp8.OK
    if "dt" in ok:
        assert f(dt=5) == fp8.ERR_INVALID_ARG
    else:
        assert f(pow2=3) == fp8.ERR_INVALID_ARG
        assert f(s=NULL) == fp8.ERR_INVALID_ARG
        assert f(s=ODD) == fp8.ERR_MISALIGNED
        assert f(ws=BAD) == fp8.ERR_MISALIGNED
        assert f(bytes=-1) == fp8.ERR_INVALID_ARG
    if "off" in ok:
        assert f(G=-1) == fp8.ERR_INVALID_ARG
        assert f(T=-1) == fp8.ERR_INVALID_ARG
        assert f(T=0) == fp8.ERR_INVALID_ARG
        assert f(off=NULL) == fp8.ERR_INVALID_ARG
        assert f(off=ODD) == fp8.ERR_MISALIGNED
        assert f(idx=ODD) == fp8.ERR_MISALIGNED
        assert f(idx=NULL) == fp8.ERR_INVALID_ARG  # rows in order need T == M_total
        assert f(T=1 << 20, K=1 << 13) == fp8.ERR_UNSUPPORTED
        assert f(G=0) == fp8.OK


def test_gated_backward_validation(L):
    f = _caller(L.fp8_gated_backward_quant, dict(dh=GOOD, gu=GOOD, dt=fp8.BF16, M=128, I=256, ld=256, pow2=0, q=GOOD,
                                                 s=GOOD, qt=GOOD, st=GOOD, qht=GOOD, sht=GOOD, stream=NULL))
    assert f(dt=4) == fp8.ERR_INVALID_ARG
    assert f(M=-128) == fp8.ERR_INVALID_ARG
    assert f(pow2=2) == fp8.ERR_INVALID_ARG
    assert f(I=200, ld=200) == fp8.ERR_UNSUPPORTED
    assert f(M=100) == fp8.ERR_UNSUPPORTED
    assert f(ld=128) == fp8.ERR_INVALID_ARG
    assert f(ld=260) == fp8.ERR_MISALIGNED
    for k in ("dh", "gu", "q", "s", "qt", "st", "qht", "sht"):
        assert f(**{k: NULL}) == fp8.ERR_INVALID_ARG  # an input, or half a pair
    assert f(q=NULL, s=NULL, qt=NULL, st=NULL, qht=NULL, sht=NULL) == fp8.ERR_INVALID_ARG
    for k in ("dh", "gu", "q", "qt", "qht"):
        assert f(**{k: BAD}) == fp8.ERR_MISALIGNED
    for k in ("s", "st", "sht"):
        assert f(**{k: ODD}) == fp8.ERR_MISALIGNED
    assert f(M=0, dh=NULL, gu=NULL) == fp8.OK


def test_grad_norm_validation(L):
    need = L.fp8fg_grad_norm_workspace(2)
    assert need > 0 and L.fp8fg_grad_norm_workspace(0) == 0
    arr = lambda t, *v: (t * len(v))(*v)
    P, N, D = (lambda *v: arr(ctypes.c_void_p, *v)), (lambda *v: arr(ctypes.c_int64, *v)), \
        (lambda *v: arr(ctypes.c_int, *v))
    good = P(0x10000, 0x20000)
    f = _caller(L.fp8fg_clip_grad_norm, dict(g=good, o=good, n=N(5, 6), d=D(0, 1), k=2, limit=1.0, norm=GOOD, ws=GOOD,
                                             bytes=need, stream=NULL))
    assert f(k=-1) == fp8.ERR_INVALID_ARG
    assert f(norm=NULL) == fp8.ERR_INVALID_ARG
    assert f(g=None) == fp8.ERR_INVALID_ARG
    assert f(o=None) == fp8.ERR_INVALID_ARG
    assert f(limit=0.0) == fp8.ERR_INVALID_ARG
    assert f(limit=float("nan")) == fp8.ERR_INVALID_ARG
    assert f(n=N(5, -1)) == fp8.ERR_INVALID_ARG
    assert f(n=N(5, 1 << 40)) == fp8.ERR_UNSUPPORTED
    assert f(d=D(0, 9)) == fp8.ERR_INVALID_ARG
    assert f(g=P(0x10000, None)) == fp8.ERR_INVALID_ARG
    assert f(o=P(0x10000, None)) == fp8.ERR_INVALID_ARG
    assert f(g=P(0x10002, 0x20000)) == fp8.ERR_MISALIGNED  # fp32 at 2 bytes
    assert f(g=P(0x10000, 0x20001)) == fp8.ERR_MISALIGNED  # bf16 at 1 byte
    assert f(bytes=need - 1) == fp8.ERR_INVALID_ARG
    assert f(ws=ODD) == fp8.ERR_MISALIGNED
    g = _caller(L.fp8fg_grad_norm, dict(g=good, n=N(5, 6), d=D(0, 1), k=2, norm=GOOD, ws=GOOD, bytes=need,
                                        stream=NULL))
    assert g(k=-1) == fp8.ERR_INVALID_ARG
    assert g(ws=NULL) == fp8.ERR_INVALID_ARG
    assert g(d=D(3, 1)) == fp8.ERR_INVALID_ARG

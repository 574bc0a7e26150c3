"""Residual addition, RMS norm and 1x128 quantisation, and the norm's gradient,
against their 64-bit formulas.

Bounds.  Forward: the sum of squares adds at most 32 elements per lane in
sequence, 6 levels of a wavefront and 16 wavefronts: 54 roundings of positive
terms, so rstd is off by half of that, one for z (each z^2 carries two halves of
z's rounding) and four for the mean, eps, root and reciprocal: 32 U.  y adds z's
rounding and two products: 35 U, taken as 40 U.  Backward: with A the sum of
|d n| over the row, the dot is off by at most (54 + 4) U A; dx follows with a
handful of roundings of each term.  dw: at most ceil(M/P) + P/32 + 32 additions
in sequence."""

import pytest
import torch

from fp8_fine_grained_amd import binding, layer
from tests.gpu_util import check_guard, guarded, say
from tests.layer_reference import U, check_close, check_quant

pytestmark = pytest.mark.gpu

REL_RSTD, REL_Y = 32 * U, 40 * U
EPS = 1e-6
# one group, one row; rows that leave wavefronts and steps part empty; every shape of the dispatch
SHAPES = [(1, 128), (3, 128), (7, 384), (2, 512), (5, 640), (33, 1024), (1, 1152), (19, 2048), (6, 2176), (2, 4096),
          (257, 4224), (1, 7168), (70, 7168), (3, 8192), (2, 8320), (2, 16384), (2, 16512), (1, 32768)]


def _inputs(M, H, dtype, seed=0, pitch=0):
    g = torch.Generator().manual_seed(seed + M * 7 + H)

    def rows(std):
        full = torch.randn((M, H + pitch), generator=g) * std
        full[torch.rand(full.shape, generator=g) < 0.001] *= 100
        return full.to(dtype)

    x, r = rows(1.0), rows(2.0)
    w = (1 + 0.1 * torch.randn(H, generator=g))
    return x, r, w


def _forward_ref(x, r, w):
    z = x.double() + (r.double() if r is not None else 0)
    rstd = 1 / torch.sqrt((z * z).mean(dim=1) + EPS)
    return z, rstd, z * rstd[:, None] * w.double()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,H", SHAPES)
def test_forward(gpu, M, H, dtype):
    say(f"norm forward {M}x{H} {dtype}")
    x, r, w = _inputs(M, H, dtype)
    for residual in (None, r):
        for pow2 in (False, True):
            wd = w if pow2 else w.to(dtype)
            z, rstd, y = _forward_ref(x, residual, wd)
            yo = torch.empty((M, H), dtype=dtype, device=gpu)
            h, q, s, rs = layer.fp8_add_rmsnorm_quant_1x128(
                x.to(gpu), wd.to(gpu), residual=None if residual is None else residual.to(gpu), eps=EPS, pow2=pow2,
                y=yo)
            what = f"{M}x{H} residual={residual is not None} pow2={pow2}"
            check_close(h, z, 0 if dtype == torch.bfloat16 else 0, what + " h", floor=U * float(z.abs().max()))
            check_close(rs, rstd, REL_RSTD, what + " rstd")
            check_close(yo, y, REL_Y, what + " y")
            check_quant(q, s, y, REL_Y, pow2, what)


def test_strided_rows_and_bounds(gpu):
    """Rows with a pitch, outputs in guarded buffers: nothing outside them is written."""
    M, H = 9, 640
    for dtype, pitch in ((torch.bfloat16, 8), (torch.float32, 4)):
        say(f"norm strided {dtype}")
        x, r, w = _inputs(M, H, dtype, pitch=pitch)
        xd, rd = x.to(gpu)[:, :H], r.to(gpu)[:, :H]
        bufs = {k: guarded(shape, dt) for k, shape, dt in (
            ("h", (M, H), dtype), ("y", (M, H), dtype), ("q", (M, H), torch.uint8), ("scales", (M, H // 128),
                                                                                     torch.float32),
            ("rstd", (M,), torch.float32))}
        layer.fp8_add_rmsnorm_quant_1x128(xd, w.to(gpu), residual=rd, eps=EPS, **{k: v for k, (_, v) in bufs.items()})
        z, rstd, y = _forward_ref(x[:, :H], r[:, :H], w)
        check_close(bufs["rstd"][1], rstd, REL_RSTD, "rstd")
        check_quant(bufs["q"][1], bufs["scales"][1], y, REL_Y)
        dx, dw = guarded((M, H), dtype), guarded((H,), torch.float32)
        layer.fp8_rmsnorm_backward(xd, rd, bufs["rstd"][1], w.to(gpu), dh=xd, dx=dx[1], dw=dw[1])
        _check_backward(x[:, :H], r[:, :H], bufs["rstd"][1].cpu(), w, x[:, :H], dx[1], dw[1], "strided")
        torch.cuda.synchronize()
        for b, _ in [*bufs.values(), dx, dw]:
            check_guard(b)


def test_zero_rows_and_extreme_values(gpu):
    """A row of zeros (zero codes, scale and gradient stay finite), rows at both
    ends of the range the squares allow, and an empty batch."""
    H = 256
    x = torch.zeros((4, H))
    x[1] = 1e18
    x[2] = 1e-18
    x[3, 5] = 3.0
    w = torch.ones(H)
    h, q, s, rstd = layer.fp8_add_rmsnorm_quant_1x128(x.to(gpu), w.to(gpu), eps=EPS)
    assert h.data_ptr() != 0 and torch.equal(h.cpu(), x)
    _, ref_rstd, y = _forward_ref(x, None, w)
    check_close(rstd, ref_rstd, REL_RSTD, "rstd")
    check_quant(q, s, y, REL_Y)
    assert torch.all(q[0] == 0) and torch.all(s[0] == 0)
    dx, dw = layer.fp8_rmsnorm_backward(torch.ones((4, H), device=gpu), x.to(gpu), rstd, w.to(gpu))
    assert torch.isfinite(dx).all() and torch.isfinite(dw).all()
    e = torch.empty((0, H), device=gpu)
    assert layer.fp8_add_rmsnorm_quant_1x128(e, w.to(gpu))[1].shape == (0, H)
    dx, dw = layer.fp8_rmsnorm_backward(e, e, torch.empty(0, device=gpu), w.to(gpu))
    assert dx.shape == (0, H) and torch.all(dw == 0)


def test_groups_below_the_normal_range(gpu):
    """Weights that leave a group's largest |y| below 448 * 2^-126: codes of value zero, no NaN,
    and the other groups as always."""
    for dtype in (torch.bfloat16, torch.float32):
        x, r, w = _inputs(3, 512, dtype)
        x[:, 5] = r[:, 5] = 0  # a zero among the tiny values
        w[:128] = 1e-38
        w[128:256] = 3e-38
        _, q, s, _ = layer.fp8_add_rmsnorm_quant_1x128(x.to(gpu), w.to(gpu), residual=r.to(gpu))
        assert torch.all(q[:, :256] & 0x7F == 0) and torch.all(s[:, :2] < 2.0 ** -126)
        y = _forward_ref(x, r, w)[2]
        check_quant(q[:, 256:].contiguous(), s[:, 2:].contiguous(), y[:, 256:].contiguous(), REL_Y, False, "others")


def test_eps_zero_and_large(gpu):
    x, _, w = _inputs(3, 256, torch.float32)
    for eps in (0.0, 10.0):
        _, q, s, rstd = layer.fp8_add_rmsnorm_quant_1x128(x.to(gpu), w.to(gpu), eps=eps)
        ref = 1 / torch.sqrt((x.double() ** 2).mean(1) + eps)
        check_close(rstd, ref, REL_RSTD, f"rstd eps={eps}")
        check_quant(q, s, x.double() * ref[:, None] * w.double(), REL_Y)


def test_not_a_number_reaches_the_codes(gpu):
    """A NaN in a row makes that row's codes NaN (0x7F/0xFF), and no other row's."""
    x, _, w = _inputs(3, 256, torch.float32)
    x[1, 7] = float("nan")
    _, q, _, rstd = layer.fp8_add_rmsnorm_quant_1x128(x.to(gpu), w.to(gpu))
    bad = (q.cpu() & 0x7F) == 0x7F
    assert bad[1].all() and not bad[0].any() and not bad[2].any()
    assert torch.isnan(rstd[1]) and torch.isfinite(rstd[0])


def _check_backward(dy, h, rstd, w, dh, dx, dw, what):
    M, H = dy.shape
    n = h.double() * rstd.double()[:, None]
    d = dy.double() * w.double()
    dot, mag = (d * n).sum(1, keepdim=True), (d * n).abs().sum(1, keepdim=True)
    ref = rstd.double()[:, None] * (d - n * dot / H) + (dh.double() if dh is not None else 0)
    floor = rstd.double()[:, None] * (8 * U * (d.abs() + (n * dot / H).abs()) + 64 * U * n.abs() * mag / H)
    if dh is not None:
        floor = floor + U * dh.double().abs()
    check_close(dx, ref, 2 * U, what + " dx", floor=floor * 1.01)
    if dw is not None:
        terms = dy.double() * n
        check_close(dw, terms.sum(0), 0, what + " dw", floor=(M + 64) * U * terms.abs().sum(0))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,H", SHAPES + [(1500, 256), (1100, 2176)])
def test_backward(gpu, M, H, dtype):
    say(f"norm backward {M}x{H} {dtype}")
    x, r, w = _inputs(M, H, dtype, seed=3)
    dy = (x.float() * 1e-3).to(dtype)
    rstd = (1 / torch.sqrt((r.double() ** 2).mean(1) + EPS)).float()
    for dh in (None, x):
        wd = w if dh is None else w.to(dtype)
        args = [t.to(gpu) for t in (dy, r, rstd, wd)]
        dx, dw = layer.fp8_rmsnorm_backward(*args, dh=None if dh is None else dh.to(gpu))
        _check_backward(dy, r, rstd, wd, dh, dx, dw, f"{M}x{H} dh={dh is not None}")
        dx2, dw2 = layer.fp8_rmsnorm_backward(*args, dh=None if dh is None else dh.to(gpu))
        assert torch.equal(dw, dw2) and torch.equal(dx, dx2), "not the same on every run"
        dx3, none = layer.fp8_rmsnorm_backward(*args, dh=None if dh is None else dh.to(gpu), need_dw=False)
        assert none is None and torch.equal(dx, dx3)


def test_backward_against_differences(gpu):
    """dx and dw against central differences of the 64-bit forward.

    f = sum(c * y): its second differences leave a relative error of about
    step^2 (1e-8), far below the fp32 bound of 1e-5 on the gradients here."""
    M, H = 2, 128
    x, _, w = _inputs(M, H, torch.float32, seed=5)
    x = x.clamp(-5, 5)
    c = torch.randn((M, H), generator=torch.Generator().manual_seed(1))

    def f(xx, ww):
        return float((c.double() * _forward_ref(xx, None, ww)[2]).sum())

    _, _, _, rstd = layer.fp8_add_rmsnorm_quant_1x128(x.to(gpu), w.to(gpu), eps=EPS)
    dx, dw = layer.fp8_rmsnorm_backward(c.to(gpu), x.to(gpu), rstd, w.to(gpu))
    step = 1e-4
    for i, j in ((0, 0), (1, 77), (0, 127)):
        e = torch.zeros((M, H), dtype=torch.float64)
        e[i, j] = step
        num = (f(x.double() + e, w) - f(x.double() - e, w)) / (2 * step)
        assert abs(num - float(dx[i, j])) <= 1e-5 * max(1.0, abs(num))
        e = torch.zeros(H, dtype=torch.float64)
        e[j] = step
        num = (f(x, w.double() + e) - f(x, w.double() - e)) / (2 * step)
        assert abs(num - float(dw[j])) <= 1e-5 * max(1.0, abs(num))


def test_other_stream_and_graph(gpu):
    """On a stream of its own (whose scratch must outlive the call), and replayed
    in a graph between eager runs on other inputs."""
    M, H = 300, 1152
    x, r, w = (t.to(gpu) for t in _inputs(M, H, torch.bfloat16))
    ref = layer.fp8_add_rmsnorm_quant_1x128(x, w, residual=r)
    ref_b = layer.fp8_rmsnorm_backward(x, ref[0], ref[3], w, dh=r)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    got = layer.fp8_add_rmsnorm_quant_1x128(x, w, residual=r, stream=st)
    got_b = layer.fp8_rmsnorm_backward(x, got[0], got[3], w, dh=r, stream=st)
    torch.empty(1 << 22, device=gpu).fill_(float("nan"))  # would land in scratch that was given back too early
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip([*ref, *ref_b], [*got, *got_b]))

    ws = torch.empty(layer.lib().fp8_rmsnorm_backward_workspace(M, H), dtype=torch.uint8, device=gpu)
    bufs = [torch.empty_like(t) for t in (*ref, *ref_b)]
    graph = torch.cuda.CUDAGraph()
    xs = x.clone()
    with torch.cuda.graph(graph):
        layer.fp8_add_rmsnorm_quant_1x128(xs, w, residual=r, h=bufs[0], q=bufs[1], scales=bufs[2], rstd=bufs[3])
        layer.fp8_rmsnorm_backward(xs, bufs[0], bufs[3], w, dh=r, dx=bufs[4], dw=bufs[5], workspace=ws)
    for k in range(4):
        xs.copy_(x * (k + 1))
        graph.replay()
        eager = layer.fp8_add_rmsnorm_quant_1x128(xs, w, residual=r)
        eager_b = layer.fp8_rmsnorm_backward(xs, eager[0], eager[3], w, dh=r)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(bufs, [*eager, *eager_b])), f"replay {k}"


def test_refusals(gpu):
    x = torch.zeros((4, 256), dtype=torch.bfloat16, device=gpu)
    w = torch.ones(256, device=gpu)
    with pytest.raises(TypeError):
        layer.fp8_add_rmsnorm_quant_1x128(x.half(), w)
    with pytest.raises(ValueError):
        layer.fp8_add_rmsnorm_quant_1x128(x, w, residual=x.float())
    with pytest.raises(ValueError):
        layer.fp8_add_rmsnorm_quant_1x128(x, w[:128])
    with pytest.raises(ValueError):
        layer.fp8_add_rmsnorm_quant_1x128(x.t(), w)
    with pytest.raises(binding.Fp8fgError) as e:
        layer.fp8_add_rmsnorm_quant_1x128(x[:, :200], w[:200])
    assert e.value.status == binding.ERR_UNSUPPORTED
    with pytest.raises(binding.Fp8fgError) as e:  # rows 8 bytes apart from 16-byte alignment
        layer.fp8_add_rmsnorm_quant_1x128(torch.zeros((4, 260), dtype=torch.bfloat16, device=gpu)[:, 4:], w)
    assert e.value.status == binding.ERR_MISALIGNED
    with pytest.raises(binding.Fp8fgError) as e:
        layer.fp8_rmsnorm_backward(x, x, torch.ones(4, device=gpu), w,
                                   workspace=torch.empty(16, dtype=torch.uint8, device=gpu))
    assert e.value.status == binding.ERR_INVALID_ARG

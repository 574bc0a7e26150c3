"""Combination of the experts' rows and its gradient, against 64-bit references."""

import pytest
import torch

from fp8_fine_grained_amd import binding
from fp8_fine_grained_amd import experts as ex
from tests import experts_reference as ref
from tests.layer_reference import U, UB, check_close, check_quant

pytestmark = pytest.mark.gpu

SIZES = [(1, 1, 8), (1, 8, 7168), (3, 2, 128), (5, 10, 648), (33, 8, 512), (100, 3, 1160), (17, 4, 4104), (64, 6, 2048),
         (7, 32, 264), (4, 8, 16512)]


def _plan(T, k, drop, seed=0):
    """Positions of T * k entries, each row once, some -1; the number of rows."""
    g = torch.Generator().manual_seed(seed)
    n = T * k
    p = torch.randperm(n, generator=g).int()
    gone = torch.rand(n, generator=g) < drop
    p[gone] = -1
    order = p[p >= 0].argsort().argsort()
    p[p >= 0] = order.int()
    return p.view(T, k), max(1, int((~gone).sum()))


def _inputs(T, k, H, dtype, drop, seed=0):
    g = torch.Generator().manual_seed(seed + 1)
    positions, R = _plan(T, k, drop, seed)
    rows = torch.randn((R, H), generator=g).to(dtype)
    base = torch.randn((T, H), generator=g).to(dtype)
    return rows, positions, torch.randn((T, k), generator=g), base


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,k,H", SIZES)
def test_combination(gpu, T, k, H, dtype):
    for drop in (0.0, 0.4, 1.0):
        rows, positions, w, base = _inputs(T, k, H, dtype, drop)
        for weights in (w, None):
            for b in (base, None):
                y = ex.combine_experts(rows.to(gpu), positions.to(gpu), None if weights is None else weights.to(gpu),
                                       base=None if b is None else b.to(gpu))
                want, size = ref.combine(rows, positions, weights, b)
                check_close(y, want, 0.0, (T, k, H, drop), floor=k * U * size)  # one rounding per place


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,k,H", SIZES)
def test_gradient(gpu, T, k, H, dtype):
    for drop in (0.0, 0.4):
        rows, positions, w, dy = _inputs(T, k, H, dtype, drop)
        R = rows.shape[0]
        for weights in (w, None):
            on = None if weights is None else weights.to(gpu)
            before = torch.full((R + 3, H), 7.0, dtype=dtype, device=gpu)  # three rows that nothing names
            more = torch.cat([rows, torch.ones((3, H), dtype=dtype)]).to(gpu)
            d, dw = ex.combine_experts_backward(dy.to(gpu), positions.to(gpu), on, rows=more, drows=before)
            want, wd, size = ref.combine_backward(dy, positions, weights, rows, R)
            assert d is before and torch.all(d[R:] == 7)
            named = ~want[:, 0].isnan()
            assert torch.all(d[:R][~named.to(gpu)] == 7)
            check_close(d[:R].cpu()[named], want[named], U, (T, k, H))
            # a lane's sum of 8 to 16 per step, steps over the row, then 6 over the lanes
            off = (dw.cpu().double() - wd).abs()
            assert torch.all(off <= (H / 32 + 16) * U * size), (T, k, H, float((off / size).max()))
            assert torch.all(dw.cpu()[(positions < 0)] == 0)
            # either alone
            d2, none = ex.combine_experts_backward(dy.to(gpu), positions.to(gpu), on, R=R + 3, need_dweights=False)
            assert none is None and torch.equal(d2[:R][named.to(gpu)], d[:R][named.to(gpu)])
            none, dw2 = ex.combine_experts_backward(dy.to(gpu), positions.to(gpu), on, rows=more, need_drows=False)
            assert none is None and torch.equal(dw, dw2)


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,k,H", [(1, 1, 128), (1, 8, 7168), (5, 10, 640), (33, 8, 512), (100, 3, 1152),
                                   (3, 2, 16512)])
def test_quantised_gradient(gpu, T, k, H, dtype, pow2):
    for drop in (0.0, 0.4):
        rows, positions, w, dy = _inputs(T, k, H, dtype, drop)
        R = rows.shape[0]
        w[0, 0] = 0.0                       # a row of zeros
        dy[0, :128] = 0.0
        q = torch.full((R + 2, H), 9, dtype=torch.uint8, device=gpu)
        s = torch.full((R + 2, H // 128), 9.0, device=gpu)
        more = torch.cat([rows, torch.ones((2, H), dtype=dtype)]).to(gpu)
        got = ex.combine_experts_backward_quant(dy.to(gpu), positions.to(gpu), w.to(gpu), rows=more, pow2=pow2, q=q,
                                                scales=s)
        want, _, _ = ref.combine_backward(dy, positions, w, rows, R)
        named = ~want[:, 0].isnan()
        assert got[0] is q and got[1] is s
        assert torch.all(q[R:] == 9) and torch.all(s[R:] == 9) and torch.all(q[:R][~named.to(gpu)] == 9)
        check_quant(q[:R].cpu()[named], s[:R].cpu()[named], want[named], U, pow2, (T, k, H))
        _, dw = ex.combine_experts_backward(dy.to(gpu), positions.to(gpu), w.to(gpu), rows=more)
        size = ref.combine_backward(dy, positions, w, rows, R)[2]
        assert torch.all((got[2] - dw).cpu().double().abs() <= 2 * (H / 32 + 16) * U * size)
        # the codes and scales are those of the plain quantiser on the same fp32 rows
        p = positions.flatten()[positions.flatten() >= 0].long()
        t = (positions.flatten() >= 0).nonzero().flatten() // k
        d = (dy.float()[t] * w.flatten()[positions.flatten() >= 0][:, None]).to(gpu)
        if d.shape[0]:
            qa, sa = binding.fp8_quant_act_1x128(d, pow2=pow2)
            assert torch.equal(q[p.to(gpu)], qa) and torch.equal(s[p.to(gpu)], sa)


def test_gradient_against_differences(gpu):
    """<y, g> as a function of one row's and one weight's entries: linear, so a difference is the gradient."""
    rows, positions, w, base = _inputs(6, 3, 64, torch.float32, 0.3)
    g = torch.randn((6, 64), generator=torch.Generator().manual_seed(9))
    d, dw = ex.combine_experts_backward(g.to(gpu), positions.to(gpu), w.to(gpu), rows=rows.to(gpu))

    def value(r, v):
        return (ref.combine(r, positions, v, base)[0] * g.double()).sum()

    at = value(rows, w)
    for t in range(6):
        for j in range(3):
            up = w.double().clone()
            up[t, j] += 1.0
            assert abs(float(value(rows, up) - at) - float(dw[t, j])) <= 64 * U * 100
            p = int(positions[t, j])
            if p >= 0:
                r = rows.double().clone()
                r[p, 5] += 1.0
                assert abs(float(value(r, w) - at) - float(d[p, 5])) <= 64 * U * 100


def test_the_gradient_of_the_dispatch(gpu):
    """Rows that were read from the tokens: their gradients added per token, ones for weights."""
    rows, positions, _, _ = _inputs(50, 4, 256, torch.bfloat16, 0.2)
    got = ex.combine_experts(rows.to(gpu), positions.to(gpu))
    want, size = ref.combine(rows, positions)
    check_close(got, want, 0.0, "dispatch", floor=4 * U * size)


def test_positions_outside_and_pitches(gpu):
    dtype = torch.bfloat16
    rows, positions, w, base = _inputs(20, 3, 256, dtype, 0.0)
    positions[3] = torch.tensor([-2 ** 31, 60, 2 ** 31 - 1], dtype=torch.int32)
    wide = torch.zeros((60, 400), dtype=dtype)
    wide[:, 8:264] = rows
    wb = torch.zeros((20, 264), dtype=dtype)
    wb[:, :256] = base
    want, size = ref.combine(rows, positions, w, base)
    y = ex.combine_experts(wide.to(gpu)[:, 8:264], positions.to(gpu), w.to(gpu), base=wb.to(gpu)[:, :256])
    check_close(y, want, 0.0, "pitch", floor=3 * U * size)
    d, dw = ex.combine_experts_backward(wb.to(gpu)[:, :256], positions.to(gpu), w.to(gpu),
                                        rows=wide.to(gpu)[:, 8:264])
    want, wd, size = ref.combine_backward(base, positions, w, rows, 60)
    named = ~want[:, 0].isnan()
    check_close(d.cpu()[named], want[named], U, "pitch gradient")
    assert torch.all((dw.cpu().double() - wd).abs() <= 24 * U * size)
    assert torch.all(dw[3] == 0)


def test_infinities_and_nan_stay_where_they_belong(gpu):
    rows, positions, w, base = _inputs(10, 2, 128, torch.float32, 0.0)
    p, q = int(positions[4, 1]), int(positions[7, 0])
    rows[p, 3], rows[q, 5] = float("nan"), float("inf")
    positions[9] = -1                     # a token whose rows are all elsewhere
    y = ex.combine_experts(rows.to(gpu), positions.to(gpu), w.to(gpu), base=base.to(gpu)).cpu()
    assert y[4, 3].isnan() and y[7, 5].isinf() and int((~y.isfinite()).sum()) == 2
    assert torch.equal(y[9], base[9])
    # a row of a dropped place is not read: NaN there does not reach the sum
    positions[4, 1] = -1
    y = ex.combine_experts(rows.to(gpu), positions.to(gpu), w.to(gpu), base=base.to(gpu)).cpu()
    assert y[4].isfinite().all()


def test_empty(gpu):
    rows = torch.ones((4, 64), device=gpu)
    none = torch.empty((0, 2), dtype=torch.int32, device=gpu)
    assert ex.combine_experts(rows, none).shape == (0, 64)
    base = torch.randn((3, 64), device=gpu)
    no_places = torch.empty((3, 0), dtype=torch.int32, device=gpu)
    assert torch.equal(ex.combine_experts(rows, no_places, base=base), base)
    assert torch.all(ex.combine_experts(rows, no_places) == 0)
    gone = torch.zeros((3, 2), dtype=torch.int32, device=gpu)
    assert torch.equal(ex.combine_experts(rows[:0], gone, base=base), base)  # no rows at all
    d, dw = ex.combine_experts_backward(base, gone, rows=rows[:0])
    assert d.shape == (0, 64) and torch.all(dw == 0)


def test_rounding_of_bf16_outputs(gpu):
    """One rounding of the fp32 sum: at most half a step."""
    rows, positions, w, base = _inputs(40, 8, 512, torch.bfloat16, 0.0)
    y = ex.combine_experts(rows.to(gpu), positions.to(gpu), w.to(gpu)).cpu().double()
    want, size = ref.combine(rows, positions, w)
    assert torch.all((y - want).abs() <= UB * want.abs() + 9 * U * size)

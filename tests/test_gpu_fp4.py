"""4-bit weights: their quantisation bit for bit, and products of few rows with them against 64-bit references.

Whole-number operands make every sum exact in fp32 whatever its order, so those products have to be equal."""

import pytest
import torch

from fp8_fine_grained_amd import binding
from fp8_fine_grained_amd import experts as ex
from tests import experts_reference as ref
from tests.layer_reference import U, UB, gated_bound, silu

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


# ------------------------------------------------------------------ quantiser
def check_quantiser(gpu, w):
    q, s = ex.fp4_quant_weight_1x32(w.to(gpu))
    rq, rs = ref.fp4_quant(w)
    assert torch.equal(s.cpu(), rs)
    assert torch.equal(q.cpu(), rq), (q.cpu() != rq).nonzero()[:4]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("N,K", [(1, 128), (3, 256), (17, 1152), (128, 7168), (513, 640)])
def test_quantiser(gpu, N, K, dtype):
    w = torch.randn((N, K), generator=torch.Generator().manual_seed(N)) * 0.02
    check_quantiser(gpu, w.to(dtype))


def test_quantiser_on_every_bf16_value_and_tie(gpu):
    """Groups with a largest value of 6 (scale 1) and every bf16 in [0, 6] and its negation."""
    v = torch.arange(0x40C1, dtype=torch.int32).to(torch.int16).view(BF16).float()  # 0 .. 6
    v = torch.cat([v, -v])
    n = (v.numel() + 30) // 31
    g = torch.zeros((n * 31,))
    g[:v.numel()] = v
    w = torch.cat([torch.full((n, 1), 6.0), g.view(n, 31)], dim=1).flatten()
    w = torch.cat([w, torch.zeros((-w.numel()) % 128)]).view(-1, 128)
    check_quantiser(gpu, w.to(BF16))
    check_quantiser(gpu, w)
    # next to every border, in fp32
    borders = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    near = torch.cat([borders, torch.nextafter(borders, torch.tensor(0.0)),
                      torch.nextafter(borders, torch.tensor(9.0))])
    row = torch.cat([torch.tensor([-6.0]), near, -near[:10]])
    check_quantiser(gpu, row.repeat(4).view(1, 128))


def test_quantiser_scales(gpu):
    """Largest values around 6 * 2^e and 2^e over the whole range, zeros, and values below it."""
    rows = []
    for e in list(range(-149, 126)):
        for m in (1.0, 1.25, 1.5, 1.5000002, 1.75, 1.9999999):
            rows.append(torch.ldexp(torch.tensor([m], dtype=torch.float64), torch.tensor(e)).float())
    top = torch.cat(rows + [torch.tensor([0.0, -0.0, 3.4028235e38, 1e-45])])
    top = top[top.isfinite()]
    top = torch.cat([top, torch.zeros((-top.numel()) % 4)])
    w = torch.randn((top.numel(), 32), generator=torch.Generator().manual_seed(0)).clamp(-1, 1).double() * \
        top.double()[:, None]
    w[:, 7] = -top
    check_quantiser(gpu, w.float().view(-1, 128))


def test_quantiser_takes_a_pitch_and_experts(gpu):
    w = torch.randn((40, 300), generator=torch.Generator().manual_seed(1)).to(gpu)
    a, b = ex.fp4_quant_weight_1x32(w[:, 4:260]), ex.fp4_quant_weight_1x32(w[:, 4:260].contiguous())
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    w = torch.randn((3, 40, 256), generator=torch.Generator().manual_seed(2)).to(gpu)
    q, s = ex.fp4_quant_weight_1x32(w)
    assert q.shape == (3, 40, 128) and s.shape == (3, 40, 8)
    for e in range(3):
        assert all(torch.equal(x, y) for x, y in zip((q[e], s[e]), ex.fp4_quant_weight_1x32(w[e])))
    assert ex.fp4_quant_weight_1x32(w[0, :0])[0].shape == (0, 128)


# ------------------------------------------------------------------ products
def _whole(shape, gen, values):
    return torch.tensor(values)[torch.randint(0, len(values), shape, generator=gen)]


def exact_operands(M, N, K, codes, seed=0, G=None):
    """x and w whose products are multiples of 2^-3 below 2^5, so that sums of 2^16 of them are exact in fp32."""
    g = torch.Generator().manual_seed(seed)
    x = _whole((M, K), g, [-2.0, -1.0, -0.5, 0.0, 0.5, 1.0, 1.5, 2.0])
    lead = (N,) if G is None else (G, N)
    q = torch.randint(0, 256, (*lead, K // 2), generator=g, dtype=torch.uint8)
    s = torch.randint(126, 129, (*lead, K // 32), generator=g, dtype=torch.uint8)
    if not codes:
        return x.to(BF16), None, q, s
    # scales that are powers of two keep the products exact
    return x.to(torch.float8_e4m3fn).view(torch.uint8), _whole((M, K // 128), g, [0.5, 1.0]), q, s


def real_operands(M, N, K, codes, seed=0, G=None):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((M, K), generator=g)
    lead = N if G is None else G * N
    q, s = ref.fp4_quant(torch.randn((lead, K), generator=g) * 0.02)
    if G is not None:
        q, s = q.view(G, N, -1), s.view(G, N, -1)
    if not codes:
        return x.to(BF16), None, q, s
    sx = x.view(M, K // 128, 128).abs().amax(dim=2) / 448
    return (x / sx.repeat_interleave(128, 1)).to(torch.float8_e4m3fn).view(torch.uint8), sx, q, s


def on(gpu, *ts):
    return [None if t is None else t.to(gpu) for t in ts]


SIZES = [(1, 1, 128), (1, 16, 256), (1, 4096, 7168), (2, 100, 640), (3, 17, 1152), (5, 33, 384), (16, 64, 2048),
         (17, 130, 896), (31, 1000, 1280), (33, 48, 128), (64, 80, 1024), (65, 256, 512), (130, 70, 1664),
         (1, 7168, 2048), (8, 2304, 18432)]


@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_whole_numbers_are_exact(gpu, M, N, K, codes):
    x, sx, w, sw = exact_operands(M, N, K, codes)
    want, _ = ref.fp4_product(ref.x_values(x, sx), ref.fp4_values(w, sw))
    xs, sxs, ws, sws = on(gpu, x, sx, w, sw)
    got = ex.fp4_gemm(xs, ws, sws, sx=sxs, out_dtype=F32)
    assert torch.equal(got.cpu().double(), want)
    got = ex.fp4_gemm(xs, ws, sws, sx=sxs)
    assert torch.equal(got.cpu(), want.float().to(BF16))


@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_products(gpu, M, N, K, codes):
    x, sx, w, sw = real_operands(M, N, K, codes)
    want, size = ref.fp4_product(ref.x_values(x, sx), ref.fp4_values(w, sw))
    xs, sxs, ws, sws = on(gpu, x, sx, w, sw)
    for dtype in (F32, BF16):
        got = ex.fp4_gemm(xs, ws, sws, sx=sxs, out_dtype=dtype).cpu().double()
        off = (got - want).abs()
        assert torch.all(off <= sum_rel(K) * size + (UB if dtype == BF16 else U) * want.abs())


def sum_rel(K):
    """Roundings of a sum over K relative to its magnitudes: exact products, added one after the other in at least
    four parts of K (K/4 and a block), each addition cut off rather than rounded at worst (2U); the parts' sum."""
    return 2 * (min(K, K / 4 + 128) + 16) * U


@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("M,I,K", [(1, 1, 128), (1, 2048, 7168), (2, 50, 640), (5, 33, 384), (16, 64, 2048),
                                   (17, 130, 896), (33, 7, 256), (65, 256, 512), (8, 1152, 2304)])
def test_gated_products(gpu, M, I, K, codes):
    for make in (exact_operands, real_operands):
        x, sx, w, sw = make(M, 2 * I, K, codes)
        if make is exact_operands:
            sw -= 4  # gates of ordinary size
        y, size = ref.fp4_product(ref.x_values(x, sx), ref.fp4_values(w, sw))
        g, u = y[:, :I], y[:, I:]
        err = sum_rel(K) * size if make is real_operands else torch.zeros_like(size)
        xs, sxs, ws, sws = on(gpu, x, sx, w, sw)
        for dtype in (F32, BF16):
            got = ex.fp4_gated_gemm(xs, ws, sws, sx=sxs, out_dtype=dtype).cpu().double()
            # the sigmoid (6 roundings) and two products
            tol = gated_bound(g, u, err[:, :I], err[:, I:], 8 * U) + (UB if dtype == BF16 else U) * (silu(g) * u).abs()
            assert torch.all((got - silu(g) * u).abs() <= tol + 2.0 ** -100)


# Rows and columns that take every workgroup shape in turn (tests/test_fp4_shapes.py).
SHAPED = [(1, 4096), (2, 7168), (1, 9600), (7, 4000), (5, 9600), (16, 4000), (13, 7168), (16, 9600), (11, 16000),
          (6, 7168), (31, 7168), (64, 7168)]


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("M,N", SHAPED)
def test_every_workgroup_shape(gpu, M, N, codes, gated):
    """Dense and over segments (all rows one expert's, after an empty one), with an odd number of 128s of K, fewer
    of them than wavefronts share K, and more than the rings hold."""
    for K in (384, 128, 2176 if N <= 7168 else 1280):
        x, sx, w, sw = exact_operands(M, N, K, codes, seed=K)
        sw -= 4 if gated else 0
        y, _ = ref.fp4_product(ref.x_values(x, sx), ref.fp4_values(w, sw))
        xs, sxs, ws, sws = on(gpu, x, sx, w, sw)
        stack = [torch.stack([torch.full_like(t, 77), t]) for t in (ws, sws)]
        offsets = torch.tensor([0, 0, M], dtype=torch.int32, device=gpu)
        if gated:
            got = ex.fp4_gated_gemm(xs, ws, sws, sx=sxs, out_dtype=F32)
            h = silu(y[:, :N // 2]) * y[:, N // 2:]
            assert torch.all((got.cpu().double() - h).abs() <= 10 * U * h.abs() + 2.0 ** -100), K
            again = ex.fp4_grouped_gated_gemm(xs, offsets, *stack, sx=sxs, out_dtype=F32)
        else:
            got = ex.fp4_gemm(xs, ws, sws, sx=sxs, out_dtype=F32)
            assert torch.equal(got.cpu().double(), y), K
            again = ex.fp4_grouped_gemm(xs, offsets, *stack, sx=sxs, out_dtype=F32)
        assert torch.equal(got, again), K


def _segments(counts):
    return torch.tensor([0, *torch.tensor(counts).cumsum(0).tolist()], dtype=torch.int32)


COUNTS = [[1], [0, 1, 0], [3, 0, 5, 16, 17, 0, 1], [0, 0, 40], [64, 0, 65, 2], [1] * 70, [0] * 65 + [9], [130, 1],
          [0, 1] * 150, [0] * 600 + [3] + [0] * 300 + [1, 2], [2] * 257]


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("counts", COUNTS)
def test_expert_segments(gpu, counts, codes, gated):
    G, M, N, K = len(counts), sum(counts), 70, 384
    T = max(1, M // 2)
    offsets = _segments(counts)
    g = torch.Generator().manual_seed(M)
    rows = torch.randint(0, T, (M,), generator=g).int()
    call = ex.fp4_grouped_gated_gemm if gated else ex.fp4_grouped_gemm
    for index in (rows, None):
        x, sx, w, sw = exact_operands(T if index is not None else M, N, K, codes, seed=M, G=G)
        sw -= 3
        xv = ref.x_values(x, sx)
        xv = xv[rows.long()] if index is not None else xv
        want = torch.cat([xv[offsets[e]:offsets[e + 1]] @ ref.fp4_values(w[e], sw[e]).t() for e in range(G)])
        if gated:
            h = silu(want[:, :N // 2]) * want[:, N // 2:]
        xs, sxs, ws, sws, o, i = on(gpu, x, sx, w, sw, offsets, index)
        got = call(xs, o, ws, sws, sx=sxs, row_index=i, out_dtype=F32).cpu().double()
        if gated:
            assert torch.all((got - h).abs() <= 10 * U * h.abs() + 2.0 ** -100)
        else:
            assert torch.equal(got, want)


def test_rows_behind_the_last_segment_stay_as_they_were(gpu):
    x, _, w, sw = exact_operands(20, 64, 256, False, G=3)
    offsets = torch.tensor([0, 4, 4, 11], dtype=torch.int32)
    xs, ws, sws, o = on(gpu, x, w, sw, offsets)
    y = torch.full((20, 64), 7.0, device=gpu)
    assert ex.fp4_grouped_gemm(xs, o, ws, sws, y=y) is y
    assert torch.all(y[11:] == 7)
    v = ref.x_values(x)
    assert torch.equal(y[:4].cpu().double(), v[:4] @ ref.fp4_values(w[0], sw[0]).t())
    assert torch.equal(y[4:11].cpu().double(), v[4:11] @ ref.fp4_values(w[2], sw[2]).t())


def test_offsets_and_indices_that_break_the_rules_stay_inside(gpu):
    """Held to the rows that are there: such rows are unspecified, and nothing outside the outputs is written."""
    x, _, w, sw = exact_operands(9, 48, 256, False, G=4)
    xs, ws, sws = on(gpu, x, w, sw)
    index = torch.tensor([-5, 100, 2 ** 31 - 1, -2 ** 31, 0, 8, 9, 3, 4], dtype=torch.int32, device=gpu)
    clamped = index.clamp(0, 8).long().cpu()
    o = torch.tensor([0, 9, 9, 9, 9], dtype=torch.int32, device=gpu)
    got = ex.fp4_grouped_gemm(xs, o, ws, sws, row_index=index, out_dtype=F32)
    assert torch.equal(got.cpu().double(), ref.x_values(x)[clamped] @ ref.fp4_values(w[0], sw[0]).t())
    for bad in ([-3, 4, 2, 50, 9], [9, 0, 0, 0, 0], [0, 2 ** 31 - 1, 5, -2 ** 31, 9], [5, 5, 5, 5, 5]):
        room = torch.full((9 + 8, 48), 7.0, device=gpu)
        ex.fp4_grouped_gemm(xs, torch.tensor(bad, dtype=torch.int32, device=gpu), ws, sws, y=room[4:13])
        assert torch.all(room == 7), bad
    # rising offsets beyond the rows are held to them
    room = torch.full((9 + 8, 48), 7.0, device=gpu)
    o = torch.tensor([-2 ** 31, -5, 4, 2 ** 31 - 1, 2 ** 31 - 1], dtype=torch.int32, device=gpu)
    ex.fp4_grouped_gemm(xs, o, ws, sws, y=room[4:13])
    v = ref.x_values(x)
    assert torch.equal(room[4:8].cpu().double(), v[:4] @ ref.fp4_values(w[1], sw[1]).t())
    assert torch.equal(room[8:13].cpu().double(), v[4:] @ ref.fp4_values(w[2], sw[2]).t())
    assert torch.all(room[:4] == 7) and torch.all(room[13:] == 7)


def test_offsets_of_many_experts_that_fall_somewhere(gpu):
    """Every expert's segment whole but for one that falls: the tiles would be more than the launch counts on."""
    G = 700
    x, _, w, sw = exact_operands(300, 48, 128, False, G=G)
    xs, ws, sws = on(gpu, x, w, sw)
    for where in (1, 255, 256, 257, 511, 512, 699):
        offsets = torch.full((G + 1,), 300, dtype=torch.int32)
        offsets[0], offsets[where] = 0, 0
        y = torch.full((300, 48), 7.0, device=gpu)
        ex.fp4_grouped_gemm(xs, offsets.to(gpu), ws, sws, y=y)
        if where == 1:  # (rises: the second expert has all rows)
            assert torch.equal(y.cpu().double(), ref.x_values(x) @ ref.fp4_values(w[1], sw[1]).t())
        else:
            assert torch.all(y == 7), where
    zigzag = torch.tensor([0, 300] * 351, dtype=torch.int32)[:G + 1]
    y = torch.full((300, 48), 7.0, device=gpu)
    ex.fp4_grouped_gemm(xs, zigzag.to(gpu), ws, sws, y=y)
    assert torch.all(y == 7)


def test_every_code_and_scale(gpu):
    """All 16 codes with every scale byte from 1 to 254, one product at a time (weights past the largest fp32 are
    infinite), and all E4M3 codes against a weight of 1."""
    K = 128
    for s0 in (1, 65, 129, 193):
        n = min(64, 255 - s0)
        codes = torch.arange(16, dtype=torch.uint8)
        w = torch.zeros((16 * n, K // 2), dtype=torch.uint8)
        sw = torch.full((16 * n, K // 32), 127, dtype=torch.uint8)
        w[:, 20] = codes.repeat(n) << 4             # element 41, in the second group
        sw[:, 1] = (torch.arange(n) + s0).repeat_interleave(16).to(torch.uint8)
        x = torch.zeros((1, K), dtype=BF16)
        x[0, 41] = 0.5 if s0 > 100 else 2.0
        want = ref.x_values(x) @ ref.fp4_values(w, sw).t()
        got = ex.fp4_gemm(*on(gpu, x, w, sw), out_dtype=F32).cpu().double()
        finite = (ref.fp4_values(w, sw).abs().amax(dim=1) < 2.0 ** 128)[None]
        assert torch.equal(got[finite], want[finite]), s0
    codes = torch.arange(256, dtype=torch.uint8)
    codes = codes[(codes & 0x7F) != 0x7F]
    x = torch.zeros((254, K), dtype=torch.uint8)
    x[:, 77] = codes
    w = torch.zeros((1, K // 2), dtype=torch.uint8)
    w[0, 38] = 2 << 4
    got = ex.fp4_gemm(*on(gpu, x, w, torch.full((1, 4), 127, dtype=torch.uint8)), sx=torch.ones((254, 1), device=gpu),
                      out_dtype=F32)
    assert torch.equal(got.cpu(), codes.view(torch.float8_e4m3fn).float()[:, None])


def test_infinities_nan_and_zero_scales(gpu):
    x, _, w, sw = exact_operands(5, 40, 256, False)
    x[1, 7], x[3, 200] = float("nan"), float("inf")
    y = ex.fp4_gemm(*on(gpu, x, w, sw), out_dtype=F32).cpu()
    assert y[1].isnan().all() and y[[0, 2, 4]].isfinite().all()   # (infinity times a code of 0 is NaN)
    assert not y[3].isfinite().any()
    x, sx, w, sw = exact_operands(5, 40, 256, True)
    sx[2] = 0.0
    y = ex.fp4_gemm(*on(gpu, x, w, sw), sx=sx.to(gpu), out_dtype=F32).cpu()
    assert torch.all(y[2] == 0) and torch.equal(y.double(), ref.x_values(x, sx) @ ref.fp4_values(w, sw).t())


def test_the_quantisers_and_the_products_together(gpu):
    """Weights and activations through the library's quantisers, then the product."""
    g = torch.Generator().manual_seed(0)
    w, x = torch.randn((300, 1024), generator=g) * 0.02, torch.randn((6, 1024), generator=g)
    q, s = ex.fp4_quant_weight_1x32(w.to(gpu))
    qx, sx = binding.fp8_quant_act_1x128(x.to(gpu))
    want, size = ref.fp4_product(ref.x_values(qx, sx), ref.fp4_values(q, s))
    got = ex.fp4_gemm(qx, q, s, sx=sx, out_dtype=F32).cpu().double()
    assert torch.all((got - want).abs() <= sum_rel(1024) * size + U * want.abs())


def test_empty(gpu):
    x, _, w, sw = on(gpu, *exact_operands(4, 32, 256, False))
    assert ex.fp4_gemm(x[:0], w, sw).shape == (0, 32)
    assert ex.fp4_gemm(x, w[:0], sw[:0]).shape == (4, 0)
    o = torch.zeros(3, dtype=torch.int32, device=gpu)
    w2, s2 = w.view(2, 16, -1), sw.view(2, 16, -1)
    y = torch.full((4, 16), 7.0, device=gpu)
    ex.fp4_grouped_gemm(x, o, w2, s2, y=y)
    assert torch.all(y == 7)
    none = torch.empty(0, dtype=torch.int32, device=gpu)
    assert ex.fp4_grouped_gated_gemm(x, o, w2, s2, row_index=none).shape == (0, 8)

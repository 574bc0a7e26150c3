"""The gated pair of block-scaled FP8 products against 64-bit arithmetic on the
same codes and scales.

Bounds.  g and u: the FP8 matrix cores' bound of tests/gpu_util.py; the exact
mode adds exact products in fp32, at most K/32 + 8 roundings in sequence and the
promotion's two per block, so (K/32 + K/64 + 8) U of the sum of magnitudes.
h: g's and u's errors through |silu'| <= 1.1, and 16 U (accurate exponential) or
64 U (hardware exponential and reciprocal: the exponent's argument g log2(e) is
off by |g| U, and |g| exp(-|g|) matters only while |g| < 20) of the product,
plus one rounding to the output type."""

import numpy as np
import pytest
import torch

from fp8_fine_grained_amd import binding, layer
from tests.gpu_util import check_guard, fp8_mfma_bound_separable, guarded, say
from tests.layer_reference import U, check_close, check_quant, gated_bound, silu

pytestmark = pytest.mark.gpu

# rows: one token, around the 16-row sub-tiles and the 128- and 256-row tiles
ROWS = [1, 2, 5, 15, 16, 17, 31, 33, 64, 65, 127, 128, 129, 200, 256, 257, 300]
# (I, K): one 1x128 group and one K block, odd multiples of 128, K blocks that leave wavefronts without work
SIZES = [(128, 128), (256, 384), (384, 896), (640, 1152)]


def _operands(gpu, M, inner, K, pow2, seed=0, G=None):
    gen = torch.Generator().manual_seed(seed + M * 31 + inner + K)
    x = torch.randn((M, K), generator=gen)
    x[torch.rand(x.shape, generator=gen) < 0.001] *= 100
    w = torch.randn(((G or 1) * 2 * inner, K), generator=gen) * (1.5 / K ** 0.5)
    qa, sa = binding.fp8_quant_act_1x128(x.to(gpu), pow2=pow2)
    qw, sw = binding.fp8_quant_weight_128x128(w.to(gpu), pow2=pow2)
    if G is not None:
        qw, sw = qw.view(G, 2 * inner, K), sw.view(G, 2 * inner // 128, K // 128)
    return qa, sa, qw, sw


def _dec(q, s, block):
    v = q.cpu().view(torch.float8_e4m3fn).double()
    s = s.cpu().double().repeat_interleave(128, dim=1)
    return v * (s.repeat_interleave(128, dim=0) if block else s)


def _reference(qa, sa, qw, sw, accum):
    """(g, u, bound of g, bound of u) in 64 bits."""
    A, W = _dec(qa, sa, False), _dec(qw, sw, True)
    K = A.shape[1]
    gu = A @ W.t()
    if accum == "exact":
        err = (A.abs() @ W.abs().t()) * (K / 32 + K / 64 + 8) * U
    else:
        err = torch.from_numpy(fp8_mfma_bound_separable(qa.cpu().numpy(), sa.cpu().numpy(), qw.cpu().numpy(),
                                                        sw.cpu().numpy(), "block"))
        err = err + (A.abs() @ W.abs().t()) * 2.0 ** -22
    n = gu.shape[1] // 2
    return gu[:, :n], gu[:, n:], err[:, :n], err[:, n:]


def _check_all(ref, accum, h=None, gu=None, quant=None, pow2=False, what=""):
    g, u, dg, du = ref
    rel = 16 * U if accum == "exact" else 64 * U
    floor = gated_bound(g, u, dg, du, rel)
    if h is not None:
        check_close(h, silu(g) * u, 0, what + " h", floor=floor)
    if gu is not None:
        check_close(gu, torch.cat([g, u], 1), 0, what + " gu", floor=torch.cat([dg, du], 1))
    if quant is not None:
        check_quant(*quant, silu(g) * u, 2 * U, pow2, what + " quant", floor=floor)


@pytest.mark.parametrize("accum", ["fp8", "exact", "scaled"])
@pytest.mark.parametrize("inner,K", SIZES)
def test_dense(gpu, inner, K, accum):
    for M in ROWS:
        say(f"gated {M}x{inner}x{K} {accum}")
        qa, sa, qw, sw = _operands(gpu, M, inner, K, accum == "scaled")
        ref = _reference(qa, sa, qw, sw, accum)
        what = f"{M}x{inner}x{K} {accum}"
        h, gu = layer.fp8_block_gated_gemm(qa, sa, qw, sw, accum=accum, save=True)
        _check_all(ref, accum, h, gu, what=what + " bf16")
        h32, gu32 = layer.fp8_block_gated_gemm(qa, sa, qw, sw, accum=accum, out_dtype=torch.float32, save=True)
        _check_all(ref, accum, h32, gu32, what=what + " f32")
        assert torch.equal(layer.fp8_block_gated_gemm(qa, sa, qw, sw, accum=accum), h), "saving changes h"
        for pow2 in (False, True):
            q, s, gq = layer.fp8_block_gated_gemm_quant(qa, sa, qw, sw, accum=accum, pow2=pow2, save=True)
            _check_all(ref, accum, gu=gq, quant=(q, s), pow2=pow2, what=what)


@pytest.mark.parametrize("accum", ["fp8", "exact", "scaled"])
@pytest.mark.parametrize("M,inner,K", [
    (1, 1024, 2048), (9, 2048, 1024), (16, 8192, 256), (20, 2048, 512), (40, 4096, 512), (64, 8192, 384),
    (100, 4096, 256), (130, 6144, 128), (300, 2048, 896), (513, 2048, 256), (1000, 4096, 128), (1030, 8192, 128)])
def test_every_workgroup_shape(gpu, M, inner, K, accum):
    """Sizes over which the choice of the workgroup's shape moves, checked on the
    rows around its edges; the quantised form with and without its workspace."""
    say(f"gated shapes {M}x{inner}x{K} {accum}")
    qa, sa, qw, sw = _operands(gpu, M, inner, K, accum == "scaled")
    h, gu = layer.fp8_block_gated_gemm(qa, sa, qw, sw, accum=accum, save=True)
    f32 = layer.fp8_block_gated_gemm(qa, sa, qw, sw, accum=accum, out_dtype=torch.float32)
    q, s, gq = layer.fp8_block_gated_gemm_quant(qa, sa, qw, sw, accum=accum, save=True)
    none = torch.empty(0, dtype=torch.uint8, device=gpu)
    q1, s1, g1 = layer.fp8_block_gated_gemm_quant(qa, sa, qw, sw, accum=accum, save=True, workspace=none)
    rows = sorted({r for r in (0, 1, 15, 16, 17, 31, 32, 63, 64, 127, 128, 255, 256, M // 2, M - 2, M - 1)
                   if 0 <= r < M})
    ref = _reference(qa[rows], sa[rows], qw, sw, accum)
    what = f"{M}x{inner}x{K} {accum}"
    _check_all(ref, accum, h[rows], gu[rows], what=what)
    _check_all(ref, accum, f32[rows], gq[rows], (q[rows], s[rows]), what=what + " f32/quant")
    _check_all(ref, accum, gu=g1[rows], quant=(q1[rows], s1[rows]), what=what + " one kernel")


def test_outputs_stay_in_their_buffers(gpu):
    for M, inner, K in ((1, 128, 256), (19, 256, 128), (130, 384, 256)):
        qa, sa, qw, sw = _operands(gpu, M, inner, K, False)
        for dt in (torch.bfloat16, torch.float32):
            h, gu = guarded((M, inner), dt), guarded((M, 2 * inner), dt)
            layer.fp8_block_gated_gemm(qa, sa, qw, sw, h=h[1], gu=gu[1])
            q, s = guarded((M, inner), torch.uint8), guarded((M, inner // 128), torch.float32)
            layer.fp8_block_gated_gemm_quant(qa, sa, qw, sw, q=q[1], scales=s[1])
            torch.cuda.synchronize()
            for b, _ in (h, gu, q, s):
                check_guard(b)


def test_large_gates(gpu):
    """Gates far on both sides: exp overflows for one, h is -0 or 0 there and g u on the other."""
    M, inner, K = 5, 128, 128
    qa, sa, qw, sw = _operands(gpu, M, inner, K, False)
    sw = sw * 1e4
    for accum in ("fp8", "exact"):
        h = layer.fp8_block_gated_gemm(qa, sa, qw, sw, accum=accum, out_dtype=torch.float32)
        assert torch.isfinite(h).all()
        _check_all(_reference(qa, sa, qw, sw, accum), accum, h, what=f"large {accum}")


@pytest.mark.parametrize("M,accum", [(1, "fp8"), (20, "exact"), (300, "fp8"), (300, "exact"), (300, "scaled")])
def test_gates_far_below_zero_quantised(gpu, M, accum):
    """The gates of a group at -88 and -123, where |h| is below the quantisers' range or zero: the
    codes are zeros, not NaN; the other group is quantised as ever.  With and without the workspace."""
    inner, K = 256, 256
    gen = torch.Generator().manual_seed(M)
    x = (1 + 0.002 * torch.rand((M, 1), generator=gen)).expand(M, K).contiguous()
    w = torch.randn((2 * inner, K), generator=gen) / K ** 0.5
    w[:128] = -88 / 256
    w[7:128:2] *= 1.4  # (320 and 448 times the scale: both exact)
    pow2 = accum == "scaled"
    qa, sa = binding.fp8_quant_act_1x128(x.to(gpu), pow2=pow2)
    qw, sw = binding.fp8_quant_weight_128x128(w.to(gpu), pow2=pow2)
    ref = _reference(qa, sa, qw, sw, accum)
    assert -88.5 < float(ref[0][:, :128].max()) < -87 and float(ref[0][:, :128].min()) < -103
    h = silu(ref[0]) * ref[1]
    assert float(h[:, :128].abs().max()) < 448 * 2.0 ** -126
    for ws in (None, torch.empty(0, dtype=torch.uint8, device=gpu)):
        q, s = layer.fp8_block_gated_gemm_quant(qa, sa, qw, sw, accum=accum, workspace=ws)
        assert torch.all(q[:, :128] & 0x7F == 0) and torch.all(s[:, 0] < 2.0 ** -126)
        floor = gated_bound(*ref, 64 * U)[:, 128:].contiguous()
        check_quant(q[:, 128:].contiguous(), s[:, 1:].contiguous(), h[:, 128:].contiguous(), 2 * U, False, "others",
                    floor=floor)


def _segments(counts):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32)


# (tokens, rows of each expert): empty first, last and middle experts, one row, tiles' edges, all rows on one expert
SEGMENTS = [(1, [1]), (16, [1] * 40), (500, [9] * 200), (2000, [700, 0, 1300]), (3, [0, 2, 0, 1]), (7, [5, 0, 0, 9, 1, 17]), (40, [0, 128, 129, 16, 0]), (300, [300, 0, 0]),
            (64, [0] * 70 + [3] * 20 + [0] * 10), (20, [0, 0])]


@pytest.mark.parametrize("accum", ["fp8", "exact", "scaled"])
@pytest.mark.parametrize("tokens,counts", SEGMENTS, ids=lambda v: str(v) if isinstance(v, int) else f"{len(v)}x{sum(v)}")
def test_grouped(gpu, tokens, counts, accum):
    inner, K = 256, 384
    G, R = len(counts), sum(counts)
    say(f"gated experts {G} rows {R} {accum}")
    qa, sa, qw, sw = _operands(gpu, tokens, inner, K, accum == "scaled", G=G)
    off = _segments(counts)
    idx = torch.randint(0, tokens, (R,), generator=torch.Generator().manual_seed(1), dtype=torch.int32)
    h, gu = layer.fp8_block_grouped_gated_gemm(qa, sa, off.to(gpu), qw, sw, row_index=idx.to(gpu), accum=accum,
                                               save=True)
    h32 = layer.fp8_block_grouped_gated_gemm(qa, sa, off.to(gpu), qw, sw, row_index=idx.to(gpu), accum=accum,
                                             out_dtype=torch.float32)
    q, s = layer.fp8_block_grouped_gated_gemm_quant(qa, sa, off.to(gpu), qw, sw, row_index=idx.to(gpu), accum=accum)
    assert h.shape == (R, inner) and q.shape == (R, inner)
    if R == 0:
        return
    li = idx.long().to(gpu)
    plain = layer.fp8_block_grouped_gated_gemm(qa[li].contiguous(), sa[li].contiguous(), off.to(gpu), qw, sw,
                                               accum=accum)
    assert torch.equal(plain, h), "rows in order differ from rows by index"
    for e in range(G):
        lo, hi = int(off[e]), int(off[e + 1])
        if lo == hi:
            continue
        ref = _reference(qa[li[lo:hi]], sa[li[lo:hi]], qw[e], sw[e], accum)
        _check_all(ref, accum, h[lo:hi], gu[lo:hi], (q[lo:hi], s[lo:hi]), what=f"expert {e}")
        _check_all(ref, accum, h32[lo:hi], what=f"expert {e} f32")


# few rows on wide experts: the small workgroup shapes, by the rows of an expert
@pytest.mark.parametrize("accum", ["fp8", "exact", "scaled"])
@pytest.mark.parametrize("counts,inner,K", [([1], 2048, 2048), ([0, 2, 0], 2048, 1024), ([22], 4096, 512),
                                            ([25], 8192, 512), ([0, 38], 8192, 512), ([40], 8192, 512)])
def test_grouped_workgroup_shapes(gpu, counts, inner, K, accum):
    G, R, tokens = len(counts), sum(counts), 16
    say(f"gated experts {counts} {inner}x{K} {accum}")
    qa, sa, qw, sw = _operands(gpu, tokens, inner, K, accum == "scaled", G=G)
    off = _segments(counts).to(gpu)
    idx = torch.randint(0, tokens, (R,), generator=torch.Generator().manual_seed(4), dtype=torch.int32).to(gpu)
    h, gu = layer.fp8_block_grouped_gated_gemm(qa, sa, off, qw, sw, row_index=idx, accum=accum, save=True)
    h32 = layer.fp8_block_grouped_gated_gemm(qa, sa, off, qw, sw, row_index=idx, accum=accum, out_dtype=torch.float32)
    q, s, gq = layer.fp8_block_grouped_gated_gemm_quant(qa, sa, off, qw, sw, row_index=idx, accum=accum, save=True)
    e = next(i for i, c in enumerate(counts) if c)  # (one expert holds every row here)
    ref = _reference(qa[idx.long()], sa[idx.long()], qw[e], sw[e], accum)
    _check_all(ref, accum, h, gu, what=f"{counts}")
    _check_all(ref, accum, h32, gq, (q, s), what=f"{counts} f32/quant")


def test_row_index_is_clamped(gpu):
    """Indices outside the tokens read a token all the same (rows unspecified, others untouched)."""
    qa, sa, qw, sw = _operands(gpu, 4, 128, 128, False, G=2)
    off = _segments([3, 3]).to(gpu)
    idx = torch.tensor([0, 1, 2, 3, 2, 1], dtype=torch.int32)
    good = layer.fp8_block_grouped_gated_gemm(qa, sa, off, qw, sw, row_index=idx.to(gpu))
    idx[1], idx[4] = -7, 1 << 20
    got = layer.fp8_block_grouped_gated_gemm(qa, sa, off, qw, sw, row_index=idx.to(gpu))
    keep = [0, 2, 3, 5]
    assert torch.equal(good[keep], got[keep])


def test_same_bits_every_run_other_stream_and_graph(gpu):
    for M, form in ((1, "bf16"), (9, "bf16"), (200, "quant")):
        qa, sa, qw, sw = _operands(gpu, M, 384, 896, False)
        call = layer.fp8_block_gated_gemm if form == "bf16" else layer.fp8_block_gated_gemm_quant
        first = call(qa, sa, qw, sw)
        first = first if isinstance(first, tuple) else (first,)
        torch.cuda.synchronize()
        again = call(qa, sa, qw, sw, stream=torch.cuda.Stream())
        again = again if isinstance(again, tuple) else (again,)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, again))
        bufs = [torch.empty_like(t) for t in first]
        kw = {"h": bufs[0]} if form == "bf16" else {"q": bufs[0], "scales": bufs[1]}
        a2 = qa.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call(a2, sa, qw, sw, **kw)
        for k in range(4):
            a2.copy_(qa.roll(k, dims=1))
            graph.replay()
            eager = call(a2, sa, qw, sw)
            eager = eager if isinstance(eager, tuple) else (eager,)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(bufs, eager)), f"replay {k}"


# ---------------------------------------------------------------- gradient
# p = sigmoid(g) carries the exponential's and the division's error, at most 4 U of
# p; 1 - p is then off by 4 U of p, which the factor 1 + g (1 - p) sees times |g|.
# dg: six more roundings of products.  du and h: four.
def _grad_reference(dh, gu):
    n = dh.shape[1]
    d, g, u = dh.double(), gu[:, :n].double(), gu[:, n:].double()
    p = torch.sigmoid(g)
    dg = d * u * p * (1 + g * (1 - p))
    floor = (d * u).abs() * p * (U * (4 * g.abs() * p + 4 * (g * (1 - p)).abs() + 16))
    return torch.cat([dg, d * g * p], 1), torch.cat([floor, 16 * U * (d * g * p).abs()], 1), g * p * u


def _grad_inputs(M, inner, dtype, seed=0, pitch=0):
    gen = torch.Generator().manual_seed(seed + M + inner)
    dh = (torch.randn((M, inner + pitch), generator=gen) * 1e-3).to(dtype)
    gu = (torch.randn((M, 2 * inner), generator=gen) * 1.7)
    gu[torch.rand(gu.shape, generator=gen) < 0.001] *= 30
    return dh, gu.to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,inner", [(1, 128), (3, 384), (17, 128), (128, 128), (129, 256), (256, 384), (384, 640),
                                     (1024, 1024)])
def test_gradient(gpu, M, inner, dtype):
    say(f"gated gradient {M}x{inner} {dtype}")
    dh, gu = _grad_inputs(M, inner, dtype)
    ref, floor, h = _grad_reference(dh, gu)
    whole = M % 128 == 0
    for pow2 in (False, True):
        r = layer.fp8_gated_backward_quant(dh.to(gpu), gu.to(gpu), pow2=pow2, columns=whole, h_columns=whole)
        check_quant(r[0], r[1], ref, 4 * U, pow2, "rows", floor)
        if whole:
            check_quant(r[2], r[3], ref.t().contiguous(), 4 * U, pow2, "columns", floor.t().contiguous())
            check_quant(r[4], r[5], h.t().contiguous(), 20 * U, pow2, "h columns")
            # any choice of outputs gives the same values
            for want in ((True, False, False), (False, True, False), (False, False, True), (True, True, False)):
                part = layer.fp8_gated_backward_quant(dh.to(gpu), gu.to(gpu), pow2=pow2, rows=want[0],
                                                      columns=want[1], h_columns=want[2])
                for k in range(6):
                    assert (part[k] is None) == (not want[k // 2])
                    assert part[k] is None or torch.equal(part[k], r[k]), f"{want} output {k}"
        else:
            assert r[2:] == (None,) * 4


def test_gradient_strides_bounds_and_extremes(gpu):
    """dh with a row pitch, gates where exp overflows or p rounds to 0 or 1, zero groups."""
    M, inner = 128, 256
    for dtype, pitch in ((torch.bfloat16, 8), (torch.float32, 4)):
        dh, gu = _grad_inputs(M, inner, dtype, pitch=pitch)
        gu[0, :inner] = 100.0
        gu[1, :inner] = -100.0
        gu[2, :inner] = -30.0
        gu[3] = 0
        dh[4] = 0
        ref, floor, h = _grad_reference(dh[:, :inner], gu)
        r = layer.fp8_gated_backward_quant(dh.to(gpu)[:, :inner], gu.to(gpu))
        # (a group whose maximum lies below 448 * 2^-126 has unspecified codes)
        live = ref.view(M, -1, 128).abs().amax(2).ge(448 * 2.0 ** -126).all(1)
        assert int((~live).sum()) <= 3
        check_quant(r[0][live.to(gpu)], r[1][live.to(gpu)], ref[live], 4 * U, False, "rows", floor[live])
        check_quant(r[2], r[3], ref.t().contiguous(), 4 * U, False, "columns", floor.t().contiguous())
        assert torch.all(r[1][4] == 0) and torch.all(r[0][4] & 0x7F == 0)


def test_gradient_at_huge_gates(gpu):
    """Gates up to the largest finite values: the sigmoid is 1 above and 0 below, and
    nothing turns into NaN on the way there.  (dh and u of the large positive ones
    are 1/2, so that every output is finite.)"""
    M, inner = 128, 256
    huge = [90.0, 1e3, 1e6, 1e10, 1e20, 1e30, 3e38]
    for dtype in (torch.bfloat16, torch.float32):
        dh, gu = _grad_inputs(M, inner, dtype)
        for i, v in enumerate(huge):
            gu[i, 5 + i] = -v                    # among ordinary values
            gu[8 + i, 128:inner] = v             # a group of one huge value
            gu[8 + i, inner + 128:] = 0.5
            dh[8 + i, 128:] = 0.5
        ref, floor, h = _grad_reference(dh, gu)
        rows = layer.fp8_gated_backward_quant(dh.to(gpu), gu.to(gpu), columns=False, h_columns=False)
        r = layer.fp8_gated_backward_quant(dh.to(gpu), gu.to(gpu))
        for q, s in (rows[:2], r[:2]):
            check_quant(q, s, ref, 4 * U, False, "rows", floor)
        check_quant(r[2], r[3], ref.t().contiguous(), 4 * U, False, "columns", floor.t().contiguous())
        check_quant(r[4], r[5], h.t().contiguous(), 20 * U, False, "h columns")


def test_gradient_groups_below_the_normal_range(gpu):
    """Gradients of saturated gates may underflow: zero codes there, no NaN, in every output."""
    M, inner = 128, 256
    for dtype in (torch.bfloat16, torch.float32):
        dh, gu = _grad_inputs(M, inner, dtype)
        gu[:, :128] = -84.0  # p about 3e-37, and dh about 1e-3
        gu[0, 3] = 0
        gu[:, inner] = 0
        q, s, qt, st, qht, sht = layer.fp8_gated_backward_quant(dh.to(gpu), gu.to(gpu))
        for codes in (q, qt, qht):
            assert not torch.any(codes & 0x7F == 0x7F)
        assert torch.all(q[1:, :128] & 0x7F == 0) and torch.all(s[1:, 0] < 2.0 ** -126)
        assert torch.all(qt[:3] & 0x7F == 0) and torch.all(st[:3] < 2.0 ** -126)
        rows = layer.fp8_gated_backward_quant(dh.to(gpu), gu.to(gpu), columns=False, h_columns=False)
        assert torch.equal(rows[0], q) and torch.equal(rows[1], s)


def test_gradient_against_differences(gpu):
    """The dequantised codes against central differences of the 64-bit activation:
    within half an E4M3 step (1/16 of the value, or 2^-10 of the scale) and 1e-6."""
    M, inner = 2, 128
    dh, gu = _grad_inputs(M, inner, torch.float32)
    dh = dh * 1e3
    q, s = layer.fp8_gated_backward_quant(dh.to(gpu), gu.to(gpu), columns=False, h_columns=False)[:2]
    s = s.cpu().double().repeat_interleave(128, 1)
    got = q.cpu().view(torch.float8_e4m3fn).double() * s

    def f(v):
        return (dh.double() * silu(v[:, :inner]) * v[:, inner:]).sum()

    step = 1e-5
    for i, j in ((0, 3), (1, 100), (0, 128 + 9), (1, 255)):
        e = torch.zeros_like(gu, dtype=torch.float64)
        e[i, j] = step
        num = float((f(gu.double() + e) - f(gu.double() - e)) / (2 * step))
        assert abs(num - float(got[i, j])) <= abs(num) / 16 + 2.0 ** -10 * float(s[i, j]) + 1e-6


def test_gradient_through_the_products(gpu):
    """dX and dW of the pair from the quantised gradient and the library's GEMMs,
    against the same products of the dequantised operands in 64 bits."""
    M, inner, K = 128, 128, 256
    gen = torch.Generator().manual_seed(9)
    x, w = torch.randn((M, K), generator=gen).to(gpu), torch.randn((2 * inner, K), generator=gen).to(gpu) / 16
    qx, sx = binding.fp8_quant_act_1x128(x)
    qw, sw, qwt, swt = binding.fp8_quant_weight_128x128_dual(w)
    dh, _ = _grad_inputs(M, inner, torch.float32)
    _, gu = layer.fp8_block_gated_gemm(qx, sx, qw, sw, accum="exact", out_dtype=torch.float32, save=True)
    q, s, qt, st, qht, sht = layer.fp8_gated_backward_quant(dh.to(gpu), gu)
    dx = binding.fp8_block_gemm(q, s, qwt, swt, accum="exact", out_dtype=torch.float32)
    qxt, sxt = binding.fp8_quant_act_1x128(x.t())
    dw = binding.fp8_block_gemm(qt, st, qxt, sxt, b_scale_mode="row", accum="exact", out_dtype=torch.float32)
    for got, a, b in ((dx, _dec(q, s, False), _dec(qwt, swt, True)), (dw, _dec(qt, st, False), _dec(qxt, sxt, False))):
        ref, mag = a @ b.t(), a.abs() @ b.abs().t()
        assert torch.all((got.cpu().double() - ref).abs() <= 32 * U * mag + 2.0 ** -140)


def test_refusals(gpu):
    with pytest.raises(binding.Fp8fgError) as e:
        layer.fp8_gated_backward_quant(torch.zeros((5, 128), device=gpu), torch.zeros((5, 256), device=gpu))
    assert e.value.status == binding.ERR_UNSUPPORTED  # transposed codes of 5 tokens
    with pytest.raises(ValueError):
        layer.fp8_gated_backward_quant(torch.zeros((5, 128), device=gpu), torch.zeros((5, 128), device=gpu))
    with pytest.raises(ValueError):
        layer.fp8_gated_backward_quant(torch.zeros((5, 128), device=gpu),
                                       torch.zeros((5, 256), dtype=torch.bfloat16, device=gpu))
    qa, sa, qw, sw = _operands(gpu, 4, 128, 256, False)
    with pytest.raises(binding.Fp8fgError) as e:
        layer.fp8_block_gated_gemm(qa, sa, qw[:128].contiguous(), sw[:1].contiguous())
    assert e.value.status == binding.ERR_UNSUPPORTED  # I = 64
    with pytest.raises(ValueError):
        layer.fp8_block_gated_gemm(qa, sa, qw, sw[:1].contiguous())
    with pytest.raises(ValueError):
        layer.fp8_block_gated_gemm(qa, sa[:, :1].contiguous(), qw, sw)
    with pytest.raises(ValueError):
        layer.fp8_block_gated_gemm(qa.t().contiguous().t(), sa, qw, sw)
    with pytest.raises(ValueError):
        layer.fp8_block_gated_gemm(qa, sa, qw, sw, h=torch.empty((4, 256), dtype=torch.bfloat16, device=gpu))
    with pytest.raises(ValueError):
        layer.fp8_block_grouped_gated_gemm(qa, sa, torch.zeros(3, dtype=torch.int32, device=gpu), qw[None], sw[None])
    with pytest.raises(ValueError):
        layer.fp8_block_gated_gemm(qa.cpu(), sa, qw, sw)

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


def _segments(counts):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32)


# (tokens, rows of each expert): empty first, last and middle experts, one row, tiles' edges, all rows on one expert
SEGMENTS = [(1, [1]), (3, [0, 2, 0, 1]), (7, [5, 0, 0, 9, 1, 17]), (40, [0, 128, 129, 16, 0]), (300, [300, 0, 0]),
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


def test_refusals(gpu):
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

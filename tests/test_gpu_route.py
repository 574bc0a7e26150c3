"""Routing of tokens to experts, its gradient and the row segments, against 64-bit references.

Choices are whole numbers and have to be equal; weights and gradients are within counted fp32 roundings."""

import pytest
import torch

from fp8_fine_grained_amd import experts as ex
from tests import experts_reference as ref
from tests.layer_reference import U, UB

pytestmark = pytest.mark.gpu

INF = float("inf")


def _logits(T, E, dtype, seed=0, std=1.0):
    return (torch.randn((T, E), generator=torch.Generator().manual_seed(seed)) * std).to(dtype)


def _bias(E, seed=1, size=0.02):
    return (torch.rand(E, generator=torch.Generator().manual_seed(seed)) - 0.5) * size


def check(gpu, z, k, what="", **kw):
    on = {n: v.to(gpu) if isinstance(v, torch.Tensor) else v for n, v in kw.items()}
    experts, weights, s = ex.route_experts(z.to(gpu), k, need_scores=True, **on)
    e, w, sr = ref.route(z, k, **kw)
    got = experts.cpu()
    assert torch.equal(got, e), (what, (got != e).nonzero()[:4].tolist(), got[(got != e).any(1)][:2],
                                 e[(got != e).any(1)][:2])
    rel = ref.rel_scores(z, kw.get("score", "sigmoid"))
    # scores of normal size to rel; smaller ones to the smallest normal number
    off = (s.cpu().double() - sr).abs()
    nan = sr.isnan()
    assert torch.equal(s.cpu().isnan(), nan), what
    assert torch.all((off <= rel * sr.abs() + 2.0 ** -126)[~nan]), (what, "scores")
    # weights: the score, the sum of up to 32 (6 roundings, each term off by rel), the quotient, the scale; a score
    # below the normal range may be lost, which a small sum of them would show: no such sums here
    off = (weights.cpu().double() - w).abs()
    nan = w.isnan()
    assert torch.equal(weights.cpu().isnan(), nan), what
    assert torch.all((off <= (2 * rel + 10 * U) * w.abs() + 2.0 ** -100)[~nan]), (what, "weights")
    return experts, weights


GROUPED = [dict(groups=8, groups_kept=4, group_terms=2), dict(groups=8, groups_kept=3, group_terms=1),
           dict(groups=4, groups_kept=4, group_terms=2)]


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 2, 2), (1, 256, 8), (37, 60, 4), (129, 160, 6), (65, 64, 8),
                                   (33, 100, 32), (64, 257, 9), (17, 512, 8), (9, 1000, 10), (5, 1024, 32),
                                   (300, 128, 1)])
def test_routing(gpu, T, E, k, dtype, score):
    z = _logits(T, E, dtype, seed=T + E)
    for bias in (None, _bias(E)):
        for renormalise in (False, True):
            check(gpu, z, k, (T, E, k), bias=bias, score=score, renormalise=renormalise, scale=2.5)
    for kw in GROUPED:
        if E % 8 == 0 and k <= kw["groups_kept"] * (E // kw["groups"]):
            for bias in (None, _bias(E)):
                check(gpu, z, k, kw, bias=bias, score=score, **kw)


@pytest.mark.parametrize("E,groups", [(72, 8), (90, 9), (96, 32), (128, 64), (256, 64), (1024, 64), (40, 2), (1000, 5),
                                      (250, 25)])
def test_group_shapes(gpu, E, groups):
    z = _logits(50, E, torch.float32, seed=E)
    for terms in (1, 2):
        for kept in (1, groups // 2 + 1):
            k = min(6, kept * (E // groups))
            for score in ("sigmoid", "softmax"):
                for bias in (None, _bias(E, size=0.3)):
                    check(gpu, z, k, (kept, terms), bias=bias, score=score, groups=groups, groups_kept=kept,
                          group_terms=terms)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_a_large_batch(gpu, score):
    z = _logits(8192, 256, torch.float32, seed=5)
    check(gpu, z, 8, bias=_bias(256), score=score, groups=8, groups_kept=4, scale=2.5)
    check(gpu, z.bfloat16(), 8, score=score)
    check(gpu, z, 8, bias=_bias(256), score=score)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_ties_go_to_the_lowest_index(gpu, score):
    E = 256
    z = torch.zeros((6, E))
    z[1] = 1.0
    z[2, 100:] = 0.5
    z[3, ::2] = -1.0
    z[4] = torch.arange(E).remainder(3).float()
    z[5] = torch.arange(E).div(32, rounding_mode="floor").remainder(2).float()
    for kw in ({}, dict(bias=torch.zeros(E)), dict(bias=torch.full((E,), 0.25)), *GROUPED,
               dict(bias=torch.zeros(E), **GROUPED[0])):
        check(gpu, z, 8, kw, score=score, **kw)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_choices_that_fp32_scores_cannot_tell(gpu, score):
    """Sums of score and bias that differ by less than their roundings in fp32, with the larger at the higher index."""
    E, T = 64, 40
    z = _logits(T, E, torch.float32, seed=7, std=0.3)
    s = ref.scores(z, score)
    b = _bias(E)
    # for every token, one expert's logit is moved (by bits) until its sum lies next to another's
    for t in range(T):
        c = s[t] + b.double()
        order = torch.sort(c, descending=True)[1]
        i, j = order[[3, 4] if t % 2 else [7, 8]].tolist()
        want = c[i] - b[j].double()
        if score == "sigmoid":
            z[t, j] = torch.log(want / (1 - want)).float()
    for bias in (b, b + 8.0, b + 3000.0):
        check(gpu, z, 8, bias=bias, score=score)
    # equal biases that swallow the scores in fp32: the order is still that of the logits
    check(gpu, z, 8, bias=torch.full((E,), 2.0 ** 24), score=score)
    # logits one bit apart
    near = torch.full((4, E), 0.7)
    near[0, 40] = torch.nextafter(torch.tensor(0.7), torch.tensor(1.0))
    near[1, 1::2] = torch.nextafter(torch.tensor(0.7), torch.tensor(1.0))
    near[2] = (torch.arange(E) * 2.0 ** -23 + 1.0)
    near[3] = -near[2]
    for kw in ({}, dict(bias=torch.zeros(E)), dict(groups=8, groups_kept=4),
               dict(bias=torch.full((E,), 0.01), groups=8, groups_kept=4)):
        check(gpu, near, 8, kw, score=score, **kw)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_masked_experts_and_tokens(gpu, score):
    E = 96
    z = _logits(12, E, torch.float32, seed=3)
    z[0] = -INF                    # nothing left
    z[1, 3:] = -INF                # fewer left than chosen
    z[2, :90] = -INF
    z[3, ::2] = -INF
    z[4, :12] = -INF               # a whole group of 8
    z[5, 1:12] = -INF              # a group with one expert
    z[6] = -3.0e38                 # the type's lowest values are numbers
    z[7, 5:] = torch.finfo(torch.float32).min
    z[8, 20] = 3.0e38
    mask = torch.ones(12, dtype=torch.bool)
    mask[[9, 11]] = False
    cut = _bias(E)
    cut[10:40] = -INF
    high = _bias(E)
    high[[7, 50, 51]] = INF
    for kw in ({}, dict(bias=_bias(E)), dict(bias=cut), dict(bias=torch.full((E,), -INF)), dict(bias=high)):
        for grouped in ({}, dict(groups=8, groups_kept=3, group_terms=2), dict(groups=8, groups_kept=3, group_terms=1)):
            for renormalise in (False, True):
                check(gpu, z, 8, (kw, grouped), score=score, mask=mask, renormalise=renormalise, **kw, **grouped)
    m = torch.zeros(12, dtype=torch.uint8)
    experts, weights = check(gpu, z, 8, score=score, mask=m)
    assert torch.all(experts == -1) and torch.all(weights == 0)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_values_that_are_not_numbers(gpu, score):
    E = 64
    z = _logits(6, E, torch.float32, seed=4)
    z[0, 10] = float("nan")
    z[1] = float("nan")
    z[2, 20] = INF
    z[3, :60] = float("nan")
    z[4, 10], z[4, 11:] = float("nan"), -INF
    for kw in ({}, dict(bias=_bias(E)), dict(groups=8, groups_kept=2)):
        check(gpu, z, 8, kw, score=score, **kw)


def test_rows_with_a_pitch_and_odd_addresses(gpu):
    wide = _logits(40, 301, torch.float32, seed=8).to(gpu)
    for dtype in (torch.float32, torch.bfloat16):
        w = wide.to(dtype)
        for lo, E in ((0, 256), (1, 256), (3, 200), (5, 60), (7, 64), (2, 128)):
            part = w[:, lo:lo + E]
            for kw in (dict(bias=_bias(E).to(gpu)), {}):
                a, b = ex.route_experts(part, 4, **kw), ex.route_experts(part.contiguous(), 4, **kw)
                assert all(torch.equal(x, y) for x, y in zip(a, b))
            dw = torch.ones((40, 4), device=gpu)
            assert torch.equal(ex.route_experts_backward(dw, a[0], part),
                               ex.route_experts_backward(dw, a[0], part.contiguous()))
    assert ex.route_experts(wide[:0], 4)[0].shape == (0, 4)


# ------------------------------------------------------------------ gradient
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 2, 2), (1, 256, 8), (333, 60, 4), (70, 64, 7), (65, 100, 32),
                                   (40, 257, 9), (17, 512, 8), (5, 1024, 32), (2000, 128, 1), (900, 256, 8)])
def test_gradient(gpu, T, E, k, dtype, score):
    z = _logits(T, E, dtype, seed=T)
    g = torch.Generator().manual_seed(2)
    experts = torch.rand((T, E), generator=g).argsort(dim=1)[:, :k].int()
    dw, ds = torch.randn((T, k), generator=g), torch.randn((T, E), generator=g) * 0.1
    for renormalise in (False, True):
        for d in (None, ds):
            check_gradient(gpu, dw, experts, z, score, renormalise, 2.5, d)


def check_gradient(gpu, dw, experts, z, score, renormalise, scale, ds):
    got = ex.route_experts_backward(dw.to(gpu), experts.to(gpu), z.to(gpu), score=score, renormalise=renormalise,
                                    scale=scale, dscores=None if ds is None else ds.to(gpu))
    assert got.dtype == z.dtype
    want, size = ref.route_backward(dw, experts, z, score, renormalise, scale, ds)
    # each term carries a score (rel), twice with renormalised weights (rel again, and the sum's); sums over up to
    # 32 places and 1024 experts (22 roundings); 1 - s and the products of the end (6)
    rel = 3 * ref.rel_scores(z, score) + 40 * U
    tol = rel * size + (UB if z.dtype == torch.bfloat16 else U) * want.abs() + 2.0 ** -100
    off = (got.cpu().double() - want).abs()
    assert torch.all(off <= tol), float((off / tol).max())
    return got


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_gradient_with_missing_repeated_and_masked_experts(gpu, score):
    z = _logits(7, 96, torch.float32, seed=9)
    z[4, 50:] = -INF
    z[5] = -INF
    z[6, ::3] = -200.0
    experts = torch.tensor([[-1, -1, -1, -1], [5, 5, 5, 5], [3, -1, 3, 95], [96, 1000, -5, 0], [50, 60, 2, -1],
                            [1, 2, 3, -1], [0, 3, 6, 9]], dtype=torch.int32)
    dw = torch.randn((7, 4), generator=torch.Generator().manual_seed(1))
    ds = torch.randn((7, 96), generator=torch.Generator().manual_seed(2))
    for renormalise in (False, True):
        for d in (None, ds):
            got = check_gradient(gpu, dw, experts, z, score, renormalise, 1.5, d)
            assert torch.all(got[5] == 0) and (d is not None or torch.all(got[0] == 0))


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renormalise", [False, True])
def test_gradient_against_differences(gpu, score, renormalise):
    """sum(weights * dw) + sum(scores * ds) as a function of the logits, by central differences in 64 bits."""
    z = _logits(4, 24, torch.float32, seed=11)
    experts, _ = ex.route_experts(z.to(gpu), 5, score=score, renormalise=renormalise, scale=2.5)
    g = torch.Generator().manual_seed(3)
    dw, ds = torch.randn((4, 5), generator=g), torch.randn((4, 24), generator=g)
    at = experts.cpu().long()

    def value(v):
        s = ref.scores(v, score)
        w = s.gather(1, at)
        w = 2.5 * (w / w.sum(dim=1, keepdim=True) if renormalise else w)
        return (w * dw.double()).sum(dim=1) + (s * ds.double()).sum(dim=1)

    got = ex.route_experts_backward(dw.to(gpu), experts, z.to(gpu), score=score, renormalise=renormalise, scale=2.5,
                                    dscores=ds.to(gpu)).cpu().double()
    h = 1e-5
    for e in range(24):
        step = torch.zeros((4, 24), dtype=torch.float64)
        step[:, e] = h
        diff = (value(z.double() + step) - value(z.double() - step)) / (2 * h)
        # the third derivative (below 10 here) times h^2 / 6, and 64-bit noise over h; fp32 roundings of terms below 10
        assert torch.all((got[:, e] - diff).abs() <= 1e-8 + 200 * U * 10)


# ------------------------------------------------------------------ segments
def check_segments(gpu, experts, G, first=0):
    offsets, rows, positions = ex.expert_segments(experts.to(gpu), G, first=first)
    o, r, p = ref.segments(experts, G, first)
    assert offsets.tolist() == o
    assert rows.tolist() == r
    assert positions.tolist() == p


@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 8, 256), (5, 3, 7), (64, 1, 2), (63, 8, 64), (257, 4, 60),
                                   (1000, 8, 1024), (1024, 2, 256), (1025, 8, 16), (4096, 8, 256), (9000, 10, 128)])
def test_segments(gpu, T, k, E):
    g = torch.Generator().manual_seed(T)
    experts = torch.randint(0, E, (T, k), generator=g).int()
    check_segments(gpu, experts, E)
    check_segments(gpu, experts, max(1, E // 3), first=E // 4)
    check_segments(gpu, torch.full_like(experts, E - 1), E)      # one expert has everything
    check_segments(gpu, torch.full_like(experts, -1), E)         # nobody has anything
    gone = torch.where(torch.rand((T, k), generator=g) < 0.3, -1, experts)
    check_segments(gpu, gone, E)


def test_segments_of_ids_outside_and_far_ranges(gpu):
    low, high = -2 ** 31, 2 ** 31 - 1
    experts = torch.tensor([[low, high, 0], [5, -1, high - 1], [high - 2, 4, low + 1]], dtype=torch.int32)
    check_segments(gpu, experts, 4)
    check_segments(gpu, experts, 6, first=2)
    check_segments(gpu, experts, 2, first=high - 2)
    offsets, rows, positions = ex.expert_segments(experts[:0].to(gpu), 5)
    assert offsets.tolist() == [0] * 6 and rows.numel() == 0 and positions.shape == (0, 3)


def test_segments_of_a_large_batch(gpu):
    """More entries than fit the units of 512: compared with a stable sort."""
    T, k, E = 150_000, 8, 200
    experts = torch.randint(-1, E, (T, k), generator=torch.Generator().manual_seed(0)).int()
    offsets, rows, positions = (t.cpu().long() for t in ex.expert_segments(experts.to(gpu), E))
    key = torch.where(experts.flatten() < 0, E, experts.flatten().long())
    order = key.argsort(stable=True)
    counts = torch.bincount(key, minlength=E + 1)[:E]
    assert offsets.tolist() == [0, *counts.cumsum(0).tolist()]
    n = int(offsets[-1])
    assert torch.equal(rows[:n], order[:n] // k) and torch.all(rows[n:] == 0)
    want = torch.full((T * k,), -1)
    want[order[:n]] = torch.arange(n)
    assert torch.equal(positions.flatten(), want)


def test_given_outputs_and_the_same_bits_again(gpu):
    z = _logits(700, 256, torch.float32).to(gpu)
    kw = dict(bias=_bias(256).to(gpu), groups=8, groups_kept=4)
    experts, weights, s = ex.route_experts(z, 8, need_scores=True, **kw)
    out = [torch.full_like(t, 7) for t in (experts, weights, s)]
    got = ex.route_experts(z, 8, experts=out[0], weights=out[1], scores=out[2], **kw)
    assert all(a is b for a, b in zip(got, out)) and all(torch.equal(a, b) for a, b in zip(out, (experts, weights, s)))
    seg = ex.expert_segments(experts, 256)
    ws = torch.empty(ex.lib().fp8fg_expert_segments_workspace(700, 8, 256), dtype=torch.uint8, device=gpu)
    out = [torch.full_like(t, 7) for t in seg]
    again = ex.expert_segments(experts, 256, offsets=out[0], row_index=out[1], positions=out[2], workspace=ws)
    assert all(a is b for a, b in zip(again, out)) and all(torch.equal(a, b) for a, b in zip(seg, out))
    dw = torch.randn((700, 8), device=gpu)
    d = ex.route_experts_backward(dw, experts, z)
    o = torch.full_like(d, 7)
    assert ex.route_experts_backward(dw, experts, z, dlogits=o) is o and torch.equal(o, d)

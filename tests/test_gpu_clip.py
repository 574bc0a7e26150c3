"""Global gradient norm and clipping against 64-bit arithmetic.

Bounds: squares are summed in 64 bits, so the norm is off by its one rounding to
fp32 (U) and an unmeasurable rest: 2 U.  c adds a division (U), an output one
product (U) and the rounding to its type."""

import math

import pytest
import torch

from fp8_fine_grained_amd import binding, layer
from tests.gpu_util import check_guard, guarded, say
from tests.layer_reference import U, check_close

pytestmark = pytest.mark.gpu

LENGTHS = [
    [1], [7], [8], [9], [8191], [8192], [8193], [1, 2, 3, 4, 5], [0], [0, 5, 0], [7168] * 5,
    [100003, 1, 8192, 16385, 3, 0, 70000],
    [257] * 121,                    # one more than a launch holds
    [33] * 500 + [90001],
    [20_000_003, 5, 8192 * 1030],   # more chunks than workgroups
]


def _grads(lengths, gpu, kinds, std=0.01, seed=0):
    g = torch.Generator(device=gpu).manual_seed(seed)
    return [(torch.randn(n, generator=g, device=gpu) * std).to(kinds[i % len(kinds)]) for i, n in enumerate(lengths)]


def _norm64(grads):
    return math.sqrt(sum(float(t.double().square().sum()) for t in grads))


@pytest.mark.parametrize("kinds", [(torch.float32,), (torch.bfloat16,), (torch.float32, torch.bfloat16)])
@pytest.mark.parametrize("lengths", LENGTHS, ids=lambda v: f"{len(v)}x{max(v)}")
def test_norm_and_clip(gpu, lengths, kinds):
    say(f"clip {len(lengths)} tensors up to {max(lengths)} {kinds}")
    grads = _grads(lengths, gpu, kinds)
    ref = _norm64(grads)
    norm = layer.grad_norm(grads)
    assert abs(float(norm) - ref) <= 2 * U * ref
    before = [t.clone() for t in grads]
    for limit in (ref / 3, ref * 2):
        if ref == 0:
            limit = 1.0
        outs = [torch.full_like(t, float("nan")) for t in grads]
        n2 = layer.clip_grad_norm(grads, limit, out=outs)
        assert torch.equal(n2, norm)
        limit32 = float(torch.tensor(limit, dtype=torch.float32))
        c = 1.0 if ref <= limit32 else limit32 / ref
        for a, b, o in zip(before, grads, outs):
            assert torch.equal(a, b), "an input was written"
            check_close(o, a.double() * c, 5 * U, f"limit {limit}")
        for t, b in zip(grads, before):
            t.copy_(b)
        layer.clip_grad_norm(grads, limit)
        assert all(torch.equal(t, o) for t, o in zip(grads, outs)), "in place differs from out of place"
        for t, b in zip(grads, before):
            t.copy_(b)


def test_views_at_odd_offsets(gpu):
    """Tensors that start at any element of a flat buffer; what lies around them stays."""
    for dtype in (torch.float32, torch.bfloat16):
        buf, flat = guarded((50_000,), dtype)
        flat.copy_(torch.randn(50_000, generator=torch.Generator().manual_seed(2)).to(dtype))
        keep = flat.clone()
        views = [flat[1:8200], flat[8203:8210], flat[8211:30_000], flat[30_005:49_999]]
        ref = _norm64(views)
        norm = layer.clip_grad_norm(views, ref / 2)
        torch.cuda.synchronize()
        assert abs(float(norm) - ref) <= 2 * U * ref
        inside = torch.zeros(50_000, dtype=torch.bool)
        for a, b in ((1, 8200), (8203, 8210), (8211, 30_000), (30_005, 49_999)):
            inside[a:b] = True
        got, was = flat.cpu(), keep.cpu()
        assert torch.equal(got[~inside], was[~inside]), "an element between the views was written"
        limit = float(torch.tensor(ref / 2, dtype=torch.float32))
        check_close(got[inside], was[inside].double() * (limit / ref), 5 * U, "views")
        check_guard(buf)


def test_extreme_values(gpu):
    """Squares beyond fp32 in both directions, infinities and NaN."""
    big = [torch.full((1000,), 1e30, device=gpu), torch.full((9,), 1e-30, device=gpu)]
    assert abs(float(layer.grad_norm(big)) / (1e30 * math.sqrt(1000)) - 1) < 1e-6
    tiny = [torch.full((1000,), 1e-30, device=gpu)]
    assert abs(float(layer.grad_norm(tiny)) / (1e-30 * math.sqrt(1000)) - 1) < 1e-6
    layer.clip_grad_norm(big, 1.0)
    assert abs(float(layer.grad_norm(big)) - 1) < 1e-5
    inf = [torch.ones(10, device=gpu), torch.tensor([1.0, float("inf")], device=gpu)]
    n = layer.clip_grad_norm(inf, 1.0)
    assert math.isinf(float(n)) and torch.all(inf[0] == 0) and float(inf[1][0]) == 0 and math.isnan(float(inf[1][1]))
    nan = [torch.ones(10, device=gpu), torch.tensor([1.0, float("nan")], device=gpu)]
    n = layer.clip_grad_norm(nan, 1.0)
    assert math.isnan(float(n)) and torch.isnan(nan[0]).all(), "a norm that is not a number must not pass unseen"


def test_empty_list(gpu):
    assert float(layer.grad_norm([])) == 0.0
    assert float(layer.clip_grad_norm([], 1.0)) == 0.0


def test_other_stream_and_graph(gpu):
    grads = _grads([70_001, 12, 8192], gpu, (torch.float32, torch.bfloat16))
    outs = [torch.empty_like(t) for t in grads]
    ref = layer.clip_grad_norm(grads, 0.5, out=outs)
    refs = [t.clone() for t in outs]
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    n = layer.clip_grad_norm(grads, 0.5, out=outs, stream=st)
    torch.empty(1 << 20, device=gpu).fill_(float("nan"))
    torch.cuda.synchronize()
    assert torch.equal(n, ref) and all(torch.equal(a, b) for a, b in zip(outs, refs))
    ws = torch.empty(layer.lib().fp8fg_grad_norm_workspace(3), dtype=torch.uint8, device=gpu)
    norm = torch.empty((), device=gpu)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.clip_grad_norm(grads, 0.5, out=outs, norm=norm, workspace=ws)
    for k in range(4):
        grads[0].mul_(1.5)
        graph.replay()
        eager = [torch.empty_like(t) for t in grads]
        en = layer.clip_grad_norm(grads, 0.5, out=eager)
        torch.cuda.synchronize()
        assert torch.equal(norm, en) and all(torch.equal(a, b) for a, b in zip(outs, eager)), f"replay {k}"


def test_refusals(gpu):
    t = torch.ones((4, 4), device=gpu)
    with pytest.raises(ValueError):
        layer.grad_norm([t.t()[:, :2]])
    with pytest.raises(TypeError):
        layer.grad_norm([t.half()])
    with pytest.raises(ValueError):
        layer.clip_grad_norm([t], 1.0, out=[])
    with pytest.raises(ValueError):
        layer.clip_grad_norm([t], 1.0, out=[t.bfloat16()])
    for bad in (0.0, -1.0, float("nan")):
        with pytest.raises(binding.Fp8fgError) as e:
            layer.clip_grad_norm([t], bad)
        assert e.value.status == binding.ERR_INVALID_ARG

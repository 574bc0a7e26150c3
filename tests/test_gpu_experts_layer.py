"""The expert layer's operators together, as they are used: streams, graphs, a training step and a server's token."""

import pytest
import torch

from fp8_fine_grained_amd import binding as fp8
from fp8_fine_grained_amd import experts as ex
from fp8_fine_grained_amd import layer
from tests import experts_reference as ref
from tests.layer_reference import U, UB, gated_bound, silu
from tests.test_gpu_fp4 import sum_rel
from tests.test_gpu_layer_streams import _leaves, _pool_of

pytestmark = pytest.mark.gpu


def _calls(gpu):
    """(name, call(**kwargs)) of every operator, with the outputs left to it."""
    g = torch.Generator().manual_seed(0)
    z = torch.randn((600, 256), generator=g).to(gpu)
    bias = torch.rand(256, generator=g).to(gpu) * 0.01
    experts, weights = ex.route_experts(z, 8, bias=bias, groups=8, groups_kept=4)
    offsets, rows, positions = ex.expert_segments(experts, 256)
    dw = torch.randn((600, 8), generator=g).to(gpu)
    x = torch.randn((600, 256), generator=g).to(gpu)
    out = torch.randn((4800, 256), generator=g).to(gpu)
    w = torch.randn((256, 64, 256), generator=g).to(gpu)
    q, s = ex.fp4_quant_weight_1x32(w)
    xb = x.bfloat16()
    return [
        ("route", lambda **k: ex.route_experts(z, 8, bias=bias, groups=8, groups_kept=4, need_scores=True, **k)),
        ("route gradient", lambda **k: ex.route_experts_backward(dw, experts, z, **k)),
        ("segments", lambda **k: ex.expert_segments(experts, 256, **k)),
        ("combine", lambda **k: ex.combine_experts(out, positions, weights, base=x, **k)),
        ("combine gradient", lambda **k: ex.combine_experts_backward(x, positions, weights, rows=out, **k)),
        ("combine gradient quantised", lambda **k: ex.combine_experts_backward_quant(x, positions, weights, rows=out,
                                                                                     **k)),
        ("fp4 quantiser", lambda **k: ex.fp4_quant_weight_1x32(w, **k)),
        ("fp4", lambda **k: ex.fp4_gemm(xb, q[0], s[0], **k)),
        ("fp4 gated", lambda **k: ex.fp4_gated_gemm(xb, q[0], s[0], **k)),
        ("fp4 experts", lambda **k: ex.fp4_grouped_gemm(xb, offsets, q, s, row_index=rows, **k)),
        ("fp4 gated experts", lambda **k: ex.fp4_grouped_gated_gemm(xb, offsets, q, s, row_index=rows, **k)),
    ]


@pytest.mark.parametrize("handle", [False, True])
def test_memory_comes_from_the_stream_of_the_call(gpu, handle, monkeypatch):
    scratch = []
    workspace = ex._workspace

    def record(*args):
        ws = workspace(*args)
        if ws[0] is not None:
            scratch.append(_pool_of(ws[0]))
        return ws

    monkeypatch.setattr(ex, "_workspace", record)
    for name, call in _calls(gpu):
        want = _leaves(call())
        torch.cuda.synchronize()
        scratch.clear()
        side = torch.cuda.Stream()
        got = _leaves(call(stream=side.cuda_stream if handle else side))
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got)), name
        assert [_pool_of(t) for t in got] == [side.cuda_stream] * len(got), name
        assert all(s == side.cuda_stream for s in scratch), name


def test_memory_still_in_use_on_the_current_stream_is_left_alone(gpu):
    """The current stream sleeps, then writes buffers that the host has already let go."""
    for name, call in _calls(gpu):
        want = _leaves(call())
        sizes = [(t.shape, t.dtype) for t in want]
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        torch.cuda._sleep(20_000_000)
        for shape, dtype in sizes:
            torch.empty(shape, dtype=dtype, device=gpu).fill_(1)
        torch.empty(1 << 20, dtype=torch.uint8, device=gpu).fill_(255)
        got = _leaves(call(stream=side))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got)), name


def test_two_calls_at_once_on_two_streams(gpu):
    for name, call in _calls(gpu):
        want = _leaves(call())
        torch.cuda.synchronize()
        sides = [torch.cuda.Stream() for _ in range(2)]
        got = [[_leaves(call(stream=s)) for s in sides] for _ in range(3)]
        torch.cuda.synchronize()
        for pair in got:
            for leaves in pair:
                assert all(torch.equal(a, b) for a, b in zip(want, leaves)), name


def test_every_call_in_a_graph(gpu):
    """Replayed several times, with the program's own eager calls and waits between: the eager results each time."""
    for name, call in _calls(gpu):
        want = _leaves(call())
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = _leaves(call())
        for _ in range(3):
            for t in got:
                t.zero_()
            graph.replay()
            eager = _leaves(call())
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(want, got)), name
            assert all(torch.equal(a, b) for a, b in zip(want, eager)), name


# ------------------------------------------------------------------ a layer in FP8 and in 4 bits
class Weights:
    def __init__(self, gpu, E, H, inner, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.E, self.H, self.inner = E, H, inner
        self.router = (torch.randn((E, H), generator=g) * H ** -0.5).to(gpu)
        self.bias = (torch.rand(E, generator=g) * 0.02).to(gpu)
        self.w13 = (torch.randn((E, 2 * inner, H), generator=g) * H ** -0.5).to(gpu)
        self.w2 = (torch.randn((E, H, inner), generator=g) * inner ** -0.5).to(gpu)
        self.route = dict(bias=self.bias, groups=4, groups_kept=2, scale=2.5)


def _token(w, x, k, q13, q2):
    """The layer for few tokens: routing, segments, the experts' gated pair and down product, combination."""
    z = x.float() @ w.router.t()
    experts, weights = ex.route_experts(z, k, **w.route)
    offsets, rows, positions = ex.expert_segments(experts, w.E)
    h = ex.fp4_grouped_gated_gemm(x, offsets, *q13, row_index=rows)
    out = ex.fp4_grouped_gemm(h, offsets, *q2)
    return ex.combine_experts(out, positions, weights, base=x), experts, weights


def _token_reference(w, x, experts, weights, q13, q2):
    """The same from the formulas in 64 bits, with the roundings of h and of the rows that their type makes, and how
    far each output may be off."""
    x = x.cpu().double()
    y, tol = x.clone(), 4 * U * x.abs()
    w13, w2 = [ref.fp4_values(*q) for q in (q13, q2)]
    for t in range(x.shape[0]):
        for e, c in zip(experts[t].tolist(), weights[t].tolist()):
            if e < 0:
                continue
            gu, size = ref.fp4_product(x[t:t + 1], w13[e])
            err = sum_rel(w.H) * size[0]
            g, u = gu[0, :w.inner], gu[0, w.inner:]
            h = silu(g) * u
            off = UB * h.abs() + gated_bound(g, u, err[:w.inner], err[w.inner:], 8 * U)
            r = w2[e] @ h
            fuzz = w2[e].abs() @ off + sum_rel(w.inner) * (w2[e].abs() @ (h.abs() + off))
            y[t] += c * r
            tol[t] += abs(c) * (fuzz + (UB + 4 * U) * (r.abs() + fuzz))  # the row's rounding, the sum's
    return y, tol + UB * (y.abs() + tol)


@pytest.mark.parametrize("T", [1, 3, 20])
def test_a_servers_tokens_in_a_graph(gpu, T):
    """Captured once, replayed on other tokens, with eager work and waits between the replays."""
    w = Weights(gpu, 16, 256, 384)
    q13, q2 = ex.fp4_quant_weight_1x32(w.w13), ex.fp4_quant_weight_1x32(w.w2)
    g = torch.Generator().manual_seed(T)
    xs = torch.randn((T, 256), generator=g).to(gpu).bfloat16()
    _token(w, xs, 3, q13, q2)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, experts, weights = _token(w, xs, 3, q13, q2)
    for k in range(4):
        xs.copy_(torch.randn((T, 256), generator=g))
        graph.replay()
        eager = _token(w, xs, 3, q13, q2)
        torch.cuda.synchronize()
        assert torch.equal(y, eager[0]) and torch.equal(experts, eager[1]) and torch.equal(weights, eager[2]), k
        want, tol = _token_reference(w, xs, experts, weights, q13, q2)
        assert torch.all((y.cpu().double() - want).abs() <= tol), k


def _step(w, x, dy, k):
    """One forward and backward pass of the layer with the experts' products in FP8: (y, dx, drouter)."""
    T = x.shape[0]
    z = x.float() @ w.router.t()
    experts, weights = ex.route_experts(z, k, **w.route)
    offsets, rows, positions = ex.expert_segments(experts, w.E)
    qx, sx = fp8.fp8_quant_act_1x128(x)
    q13 = [fp8.fp8_quant_weight_128x128_dual(m) for m in w.w13]
    q2 = [fp8.fp8_quant_weight_128x128_dual(m) for m in w.w2]

    def stack(q, i):
        return torch.stack([t[i] for t in q])

    h, gu = layer.fp8_block_grouped_gated_gemm(qx, sx, offsets, stack(q13, 0), stack(q13, 1), row_index=rows, save=True)
    qh, sh = fp8.fp8_quant_act_1x128(h)
    out = fp8.fp8_block_grouped_gemm(qh, sh, offsets, stack(q2, 0), stack(q2, 1))
    y = ex.combine_experts(out, positions, weights, base=x)
    # backward
    q, s, dweights = ex.combine_experts_backward_quant(dy, positions, weights, rows=out)
    dh = fp8.fp8_block_grouped_gemm(q, s, offsets, stack(q2, 2), stack(q2, 3))
    q, s = layer.fp8_gated_backward_quant(dh, gu, columns=False, h_columns=False)[:2]
    drows = fp8.fp8_block_grouped_gemm(q, s, offsets, stack(q13, 2), stack(q13, 3))
    dz = ex.route_experts_backward(dweights, experts, z, scale=2.5)
    dx = ex.combine_experts(drows, positions, base=dy).float() + dz @ w.router
    assert T * k == rows.numel()
    return y, dx, dz.t() @ x.float()


def test_a_training_step_of_the_layer(gpu):
    """Outputs and gradients against automatic differentiation of the formulas in 64 bits, as far as FP8 allows."""
    w = Weights(gpu, 8, 256, 256)
    T, k = 96, 2
    g = torch.Generator().manual_seed(1)
    x, dy = (torch.randn((T, 256), generator=g).to(gpu).bfloat16() for _ in range(2))
    y, dx, drouter = _step(w, x, dy, k)
    xr = x.cpu().double().requires_grad_()
    router = w.router.cpu().double().requires_grad_()
    z = xr @ router.t()
    experts, _, _ = ref.route(z.detach().float(), k, bias=w.bias, groups=4, groups_kept=2, scale=2.5)
    assert torch.equal(experts, ex.route_experts(x.float() @ w.router.t(), k, **w.route)[0].cpu())
    s = torch.sigmoid(z).gather(1, experts.long())
    weights = 2.5 * s / s.sum(dim=1, keepdim=True)
    w13, w2 = w.w13.cpu().double(), w.w2.cpu().double()
    rows = []
    for t in range(T):
        total = xr[t]
        for j in range(k):
            e = int(experts[t, j])
            gu = w13[e] @ xr[t]
            total = total + weights[t, j] * (w2[e] @ (torch.nn.functional.silu(gu[:256]) * gu[256:]))
        rows.append(total)
    yr = torch.stack(rows)
    yr.backward(dy.cpu().double())
    for got, want in ((y, yr.detach()), (dx, xr.grad), (drouter, router.grad)):
        got = got.cpu().double()
        # an E4M3 rounding of a value m 2^e, m in [1, 2), is off by up to 2^(e - 4): an rms of 2^-4 / sqrt(3) against
        # one of sqrt(7 / 3) for m, 2.4%; up to seven operands in a chain, half as much again for their spread
        assert float((got - want).norm() / want.norm()) <= 0.024 * 7 ** 0.5 * 1.5


def test_two_graphs_do_not_share_scratch(gpu):
    """Two captured calls whose workspaces come from their graphs' own memory, replayed in turn and at once."""
    g = torch.Generator().manual_seed(3)
    ids = [torch.randint(0, 64, (3000, 8), generator=g).int().to(gpu) for _ in range(2)]
    want = [ex.expert_segments(i, 64) for i in ids]
    graphs, got = [], []
    for i in ids:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got.append(ex.expert_segments(i, 64))
        graphs.append(graph)
    sides = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(4):
        for s, graph in zip(sides, graphs):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


# ------------------------------------------------------------------ operands past 32 bits
def test_rows_past_four_billion_elements(gpu):
    """Rows at both ends of 2^32 elements (9 GB of bf16), few of them named."""
    H, R = 8192, (1 << 19) + 40
    rows = torch.empty((R, H), dtype=torch.bfloat16, device=gpu)
    named = torch.tensor([0, R - 1, 1 << 18, R - 40, (1 << 18) + 1, R - 2], dtype=torch.int32)
    gen = torch.Generator().manual_seed(0)
    small = torch.randn((6, H), generator=gen).bfloat16()
    rows[named.long().to(gpu)] = small.to(gpu)
    positions = named.view(3, 2)
    w = torch.randn((3, 2), generator=gen)
    local = torch.arange(6, dtype=torch.int32).view(3, 2)
    y = ex.combine_experts(rows, positions.to(gpu), w.to(gpu))
    assert torch.equal(y, ex.combine_experts(small.to(gpu), local.to(gpu), w.to(gpu)))
    dy = torch.randn((3, H), generator=gen).bfloat16().to(gpu)
    d, dw = ex.combine_experts_backward(dy, local.to(gpu), w.to(gpu), rows=small.to(gpu))
    q, s, _ = ex.combine_experts_backward_quant(dy, local.to(gpu), w.to(gpu), rows=small.to(gpu))
    q2, s2, dw2 = ex.combine_experts_backward_quant(dy, positions.to(gpu), w.to(gpu), rows=rows)
    at = named.long().to(gpu)
    assert torch.equal(q2[at], q) and torch.equal(s2[at], s) and torch.equal(dw2, dw)
    del q2, s2
    d2, dw2 = ex.combine_experts_backward(dy, positions.to(gpu), w.to(gpu), rows=rows)
    assert torch.equal(d2[at], d) and torch.equal(dw2, dw)


def test_weights_past_four_gigabytes(gpu):
    """The last experts of a stack of 4.6 GB of codes, and the quantiser writing there."""
    G, N, K = 320, 4096, 7168
    q = torch.empty((G, N, K // 2), dtype=torch.uint8, device=gpu)
    s = torch.full((G, N, K // 32), 120, dtype=torch.uint8, device=gpu)
    g = torch.Generator(device=gpu).manual_seed(0)
    for e in (0, 1, G - 2, G - 1):
        q[e] = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device=gpu, generator=g)
    counts = torch.zeros(G, dtype=torch.int32)
    counts[[0, 1, G - 2, G - 1]] = torch.tensor([1, 2, 17, 3], dtype=torch.int32)
    offsets = torch.cat([torch.zeros(1, dtype=torch.int32), counts.cumsum(0).int()]).to(gpu)
    x = torch.randn((23, K), device=gpu, generator=g).bfloat16()
    got = ex.fp4_grouped_gemm(x, offsets, q, s)
    lo = 0
    for e, n in ((0, 1), (1, 2), (G - 2, 17), (G - 1, 3)):
        # (not bit for bit those of a dense call, whose workgroups may divide K otherwise)
        want, size = ref.fp4_product(ref.x_values(x[lo:lo + n]), ref.fp4_values(q[e], s[e]))
        off = (got[lo:lo + n].cpu().double() - want).abs()
        assert torch.all(off <= sum_rel(K) * size + UB * want.abs()), e
        lo += n
    del q, s
    w = torch.empty((9 * 65536 + 8, 8192), dtype=torch.bfloat16, device=gpu)  # 9.7 GB, 2.4 GB of codes
    w[-8:] = torch.randn((8, 8192), device=gpu, generator=g)
    w[:8] = w[-8:]
    w[8:-8].fill_(1.0)
    q, s = ex.fp4_quant_weight_1x32(w)
    assert torch.equal(q[-8:], q[:8]) and torch.equal(s[-8:], s[:8])
    assert bool((q[8:-8] == 0x66).all()) and bool((s[8:-8] == 125).all())

"""Calls on a stream that is not the current one.

Memory that such a call allocates, outputs and scratch, has to come from its own stream's
pool: a block that the current stream's queued work still uses may already be free on the
host, and the other stream does not wait for that work."""

import pytest
import torch

from fp8_fine_grained_amd import layer
from tests.test_gpu_gated import _operands

pytestmark = pytest.mark.gpu


def _pool_of(t):
    """The stream whose pool the memory of t was allocated from."""
    at = t.data_ptr()
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= at < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not the allocator's memory")


def _calls(gpu):
    """(name, call(**kwargs)) of every operator, with the outputs left to it."""
    g = torch.Generator().manual_seed(0)
    x, r = (torch.randn((256, 640), generator=g).to(gpu) for _ in range(2))
    w = torch.rand(640, generator=g).to(gpu) + 0.5
    rstd = 1 / torch.sqrt(r.square().mean(1) + 1e-6)
    qa, sa, qw, sw = _operands(gpu, 40, 1024, 1024, False)
    off = torch.tensor([0, 17, 40], dtype=torch.int32, device=gpu)
    ge = _operands(gpu, 40, 256, 384, False, G=2)
    dh, gu = x[:128, :256].contiguous(), torch.randn((128, 512), generator=g).to(gpu)
    grads = [x.flatten(), r.flatten()]
    outs = [torch.empty_like(t) for t in grads]
    return [
        ("norm", lambda **k: layer.fp8_add_rmsnorm_quant_1x128(x, w, residual=r, **k)),
        ("norm gradient", lambda **k: layer.fp8_rmsnorm_backward(x, r, rstd, w, **k)),
        ("gated", lambda **k: layer.fp8_block_gated_gemm(qa, sa, qw, sw, save=True, **k)),
        ("gated quantised", lambda **k: layer.fp8_block_gated_gemm_quant(qa, sa, qw, sw, save=True, **k)),
        ("experts", lambda **k: layer.fp8_block_grouped_gated_gemm(ge[0], ge[1], off, ge[2], ge[3], **k)),
        ("experts quantised", lambda **k: layer.fp8_block_grouped_gated_gemm_quant(ge[0], ge[1], off, ge[2], ge[3],
                                                                                   **k)),
        ("gated gradient", lambda **k: layer.fp8_gated_backward_quant(dh, gu, **k)),
        ("gradient norm", lambda **k: layer.grad_norm(iter(grads), **k)),
        ("clipping", lambda **k: layer.clip_grad_norm(iter(grads), 0.5, out=iter(outs), **k)),
    ]


def _leaves(v):
    return [t for t in (v if isinstance(v, tuple) else (v,)) if t is not None]


@pytest.mark.parametrize("handle", [False, True])
def test_memory_comes_from_the_stream_of_the_call(gpu, handle, monkeypatch):
    scratch = []
    workspace = layer._workspace

    def record(*args):
        ws = workspace(*args)
        if ws[0] is not None:
            scratch.append(_pool_of(ws[0]))
        return ws

    monkeypatch.setattr(layer, "_workspace", record)
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
        assert torch.cuda.current_stream().cuda_stream != side.cuda_stream


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


def test_results_are_kept_for_the_stream_that_is_current_outside(gpu):
    """A result dropped while the outer stream still reads it is not handed out to the side stream."""
    side = torch.cuda.Stream()
    name, call = _calls(gpu)[0]
    torch.cuda.synchronize()
    h = call(stream=side)[0]
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(20_000_000)
    copy = h.clone()
    want = call()[0]
    at, n = h.data_ptr(), h.shape
    del h
    with torch.cuda.stream(side):
        again = torch.empty(n, device=gpu)
        assert again.data_ptr() != at
        again.fill_(float("nan"))
    torch.cuda.synchronize()
    assert torch.equal(copy, want)


def test_given_outputs_and_the_current_stream_itself(gpu):
    """Outputs that the caller passes in are used as they are, and naming the current stream changes nothing."""
    qa, sa, qw, sw = _operands(gpu, 40, 256, 384, False)
    want = layer.fp8_block_gated_gemm(qa, sa, qw, sw)
    here = torch.cuda.current_stream()
    assert torch.equal(layer.fp8_block_gated_gemm(qa, sa, qw, sw, stream=here), want)
    side = torch.cuda.Stream()
    out = torch.zeros_like(want)
    side.wait_stream(here)
    assert layer.fp8_block_gated_gemm(qa, sa, qw, sw, h=out, stream=side) is out
    side.synchronize()
    assert torch.equal(out, want)


def test_capture_with_a_forked_stream(gpu):
    """Recorded into a graph on a stream forked from the capturing one; every replay against the eager call."""
    g = torch.Generator().manual_seed(1)
    x, w = torch.randn((200, 384), generator=g).to(gpu), torch.rand(384, generator=g).to(gpu)
    xs = x.clone()
    side = torch.cuda.Stream()
    layer.fp8_add_rmsnorm_quant_1x128(xs, w)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        got = layer.fp8_add_rmsnorm_quant_1x128(xs, w, stream=side)
        here.wait_stream(side)
    for k in range(4):
        xs.copy_(x * (k + 1))
        graph.replay()
        want = layer.fp8_add_rmsnorm_quant_1x128(xs, w)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got[1:], want[1:])), f"replay {k}"


def test_nothing_on_the_gpu(gpu):
    with pytest.raises(ValueError):
        layer.fp8_add_rmsnorm_quant_1x128(torch.zeros((1, 128)), torch.ones(128), stream=torch.cuda.Stream())
    side = torch.cuda.Stream()
    norm = layer.grad_norm([], stream=side)
    side.synchronize()
    assert float(norm) == 0.0

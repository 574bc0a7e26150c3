"""Quantisers and GEMMs called on a stream that is not the current one: their outputs come from
that stream's memory, not from blocks that the current stream's queued work may still use."""

import pytest
import torch

from fp8_fine_grained_amd import binding as fp8
from tests.test_gpu_layer_streams import _leaves, _pool_of

pytestmark = pytest.mark.gpu


def _calls(gpu):
    g = torch.Generator().manual_seed(0)
    x, w = torch.randn((256, 384), generator=g).to(gpu), torch.randn((512, 384), generator=g).to(gpu)
    qa, sa = fp8.fp8_quant_act_1x128(x)
    qb, sb = fp8.fp8_quant_weight_128x128(w)
    off = torch.tensor([0, 100, 256], dtype=torch.int32, device=gpu)
    idx = torch.arange(256, dtype=torch.int32, device=gpu).flip(0)
    experts = (qb.view(2, 256, 384), sb.view(2, 2, 3))
    return [
        ("activations", lambda **k: fp8.fp8_quant_act_1x128(x, **k)),
        ("weights", lambda **k: fp8.fp8_quant_weight_128x128(w, **k)),
        ("both", lambda **k: fp8.fp8_quant_act_weight(x, w, **k)),
        ("one scale", lambda **k: fp8.fp8_quant_per_tensor(x, **k)),
        ("weights both ways", lambda **k: fp8.fp8_quant_weight_128x128_dual(w, **k)),
        ("product", lambda **k: fp8.fp8_block_gemm(qa, sa, qb, sb, **k)),
        ("exact product", lambda **k: fp8.fp8_block_gemm(qa, sa, qb, sb, accum="exact", **k)),
        ("quantised product", lambda **k: fp8.fp8_block_gemm_quant(qa, sa, qb, sb, **k)),
        ("experts", lambda **k: fp8.fp8_block_grouped_gemm(qa, sa, off, *experts, **k)),
        ("experts by index", lambda **k: fp8.fp8_block_grouped_gemm_gather(qa, sa, idx, off, *experts, **k)),
    ]


@pytest.mark.parametrize("handle", [False, True])
def test_outputs_come_from_the_stream_of_the_call(gpu, handle):
    for name, call in _calls(gpu):
        want = _leaves(call())
        sizes = [(t.shape, t.dtype) for t in want]
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        torch.cuda._sleep(20_000_000)
        for shape, dtype in sizes:  # written late, and free on the host at once
            torch.empty(shape, dtype=dtype, device=gpu).fill_(1)
        got = _leaves(call(stream=side.cuda_stream if handle else side))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got)), name
        assert [_pool_of(t) for t in got] == [side.cuda_stream] * len(got), name


def test_given_outputs(gpu):
    name, call = _calls(gpu)[5]
    want, out = call(), torch.zeros((256, 512), dtype=torch.bfloat16, device=gpu)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert call(y=out, stream=side) is out
    side.synchronize()
    assert torch.equal(out, want)

"""The expert layer's operators refuse tensors of two GPUs, and of none, before anything is launched, and so they
refuse tensors of wrong types and shapes.

Needs no GPU: the tensors are fake ones, which have a device but no memory."""

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

from fp8_fine_grained_amd import binding, experts, layer

BF16, F32, U8, I32, BOOL = torch.bfloat16, torch.float32, torch.uint8, torch.int32, torch.bool

DENSE = {"x": ((4, 256), U8), "sx": ((4, 2), F32), "w": ((96, 128), U8), "sw": ((96, 8), U8)}
GROUPED = {**DENSE, "w": ((3, 96, 128), U8), "sw": ((3, 96, 8), U8), "offsets": ((4,), I32), "row_index": ((4,), I32)}
GRAD = {"dy": ((4, 256), BF16), "positions": ((4, 2), I32), "weights": ((4, 2), F32), "rows": ((7, 256), BF16),
        "dweights": ((4, 2), F32)}
CALLS = {
    "route": (experts.route_experts, dict(
        logits=((4, 64), F32), k=2, bias=((64,), F32), mask=((4,), BOOL), experts=((4, 2), I32),
        weights=((4, 2), F32), scores=((4, 64), F32))),
    "route gradient": (experts.route_experts_backward, dict(
        dweights=((4, 2), F32), experts=((4, 2), I32), logits=((4, 64), F32), dscores=((4, 64), F32),
        dlogits=((4, 64), F32))),
    "segments": (experts.expert_segments, dict(
        experts=((4, 2), I32), G=8, offsets=((9,), I32), row_index=((8,), I32), positions=((4, 2), I32),
        workspace=((1 << 16,), U8))),
    "combine": (experts.combine_experts, dict(
        rows=((7, 256), BF16), positions=((4, 2), I32), weights=((4, 2), F32), base=((4, 256), BF16),
        y=((4, 256), BF16))),
    "combine gradient": (experts.combine_experts_backward, {**GRAD, "drows": ((7, 256), BF16)}),
    "combine gradient quantised": (experts.combine_experts_backward_quant, {
        **GRAD, "q": ((7, 256), U8), "scales": ((7, 2), F32)}),
    "fp4 quantiser": (experts.fp4_quant_weight_1x32, dict(
        w=((96, 256), F32), q=((96, 128), U8), scales=((96, 8), U8))),
    "fp4": (experts.fp4_gemm, {**DENSE, "y": ((4, 96), BF16)}),
    "fp4 gated": (experts.fp4_gated_gemm, {**DENSE, "h": ((4, 48), BF16)}),
    "fp4 experts": (experts.fp4_grouped_gemm, {**GROUPED, "y": ((4, 96), BF16)}),
    "fp4 gated experts": (experts.fp4_grouped_gated_gemm, {**GROUPED, "h": ((4, 48), BF16)}),
}


def _made(name, device):
    fn, spec = CALLS[name]
    return fn, {k: torch.empty(v[0], dtype=v[1], device=device) if isinstance(v, tuple) else v
                for k, v in spec.items()}


@pytest.fixture
def no_library(monkeypatch):
    monkeypatch.setattr(experts, "lib", lambda: pytest.fail("reached the library"))
    monkeypatch.setattr(experts, "_lib", None)
    monkeypatch.setattr(layer, "_current_gpu", lambda: 0)


@pytest.mark.parametrize("other", ["cuda:1", "cpu"])
@pytest.mark.parametrize("name", CALLS)
def test_one_tensor_on_another_device(name, other, no_library):
    with FakeTensorMode():
        fn, args = _made(name, "cuda:0")
        _, moved = _made(name, other)
        for k, v in args.items():
            if isinstance(v, torch.Tensor):
                with pytest.raises(ValueError, match="one GPU"):
                    fn(**{**args, k: moved[k]})
        if other == "cpu":
            with pytest.raises(ValueError, match="one GPU"):
                fn(**moved)


@pytest.mark.parametrize("name", CALLS)
def test_another_gpu_than_the_current_one_is_made_current(name, monkeypatch):
    """The kernels have to be launched with the tensors' GPU current."""
    entered = []

    class Guard:
        def __init__(self, device):
            self.device = device

        def __enter__(self):
            entered.append(self.device)
            monkeypatch.setattr(layer, "_current_gpu", lambda: self.device)

        def __exit__(self, *a):
            pass

    class Reached(Exception):
        pass

    def reached(*a, **k):
        raise Reached

    monkeypatch.setattr(layer, "_current_gpu", lambda: 0)
    monkeypatch.setattr(torch.cuda, "device", Guard)
    for inner in ("_rows", "_fp4_operands"):  # the checks that come next
        monkeypatch.setattr(experts, inner, reached)
    with FakeTensorMode():
        fn, args = _made(name, "cuda:1")
        with pytest.raises(Reached):
            fn(**args)
    assert entered == [1]


@pytest.mark.parametrize("name", CALLS)
def test_wrong_types_shapes_and_strides(name, no_library):
    """Every tensor in turn: another type, a row more, a column more, and columns apart from each other."""
    free = {"route": {"logits": "tc"}, "route gradient": {"logits": "t"}, "fp4 quantiser": {"w": "t"},
            "combine": {"rows": "r"}}
    for k, v in CALLS[name][1].items():
        if not isinstance(v, tuple):
            continue
        shape, dtype = v
        may = free.get(name, {}).get(k, "")
        if k == "workspace":
            continue
        with FakeTensorMode():
            fn, args = _made(name, "cuda:0")

            def t(shape, dtype=dtype):
                return torch.empty(shape, dtype=dtype, device="cuda:0")

            outputs = {"y", "h"} if name.startswith("fp4") else set()
            wrong = [] if k in outputs or "t" in may else [t(shape, torch.int16)]
            if len(shape) == 2 and "r" not in may:
                wrong.append(t((shape[0] + 1, shape[1])))
            if "c" not in may and not (name == "combine" and k == "rows"):
                wrong.append(t((*shape[:-1], shape[-1] + 1)))
            wrong.append(t((*shape[:-1], 2 * shape[-1]))[..., ::2])
            for w in wrong:
                with pytest.raises((ValueError, TypeError, binding.Fp8fgError)):
                    fn(**{**args, k: w})

"""The layer operators refuse tensors of two GPUs, and of none, before anything is launched.

Needs no GPU: the tensors are fake ones, which have a device but no memory."""

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

from fp8_fine_grained_amd import layer

BF16, F32, U8, I32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32


def _norm(t):
    return layer.fp8_add_rmsnorm_quant_1x128, dict(
        x=t((4, 256), BF16), weight=t((256,), F32), residual=t((4, 256), BF16), h=t((4, 256), BF16),
        y=t((4, 256), BF16), q=t((4, 256), U8), scales=t((4, 2), F32), rstd=t((4,), F32))


def _norm_gradient(t):
    return layer.fp8_rmsnorm_backward, dict(
        dy=t((4, 256), BF16), h=t((4, 256), BF16), rstd=t((4,), F32), weight=t((256,), F32), dh=t((4, 256), BF16),
        dx=t((4, 256), BF16), dw=t((256,), F32), workspace=t((1 << 16,), U8))


GATED = {"a": ((4, 256), U8), "sa": ((4, 2), F32), "w": ((256, 256), U8), "sw": ((2, 2), F32)}
QUANT = {"q": ((4, 128), U8), "scales": ((4, 1), F32), "gu": ((4, 256), BF16), "workspace": ((1 << 16,), U8)}
PLAIN = {"h": ((4, 128), BF16), "gu": ((4, 256), BF16)}
EXPERTS = {**GATED, "w": ((3, 256, 256), U8), "sw": ((3, 2, 2), F32), "offsets": ((4,), I32), "row_index": ((4,), I32)}


def _of(fn, spec):
    return lambda t: (fn, {k: t(*v) for k, v in spec.items()})


def _clip(t):
    return layer.clip_grad_norm, dict(grads=[t((5,), F32), t((7,), BF16)], max_norm=1.0,
                                      out=[t((5,), F32), t((7,), BF16)], norm=t((), F32), workspace=t((1 << 14,), U8))


def _grad_norm(t):
    return layer.grad_norm, dict(grads=[t((5,), F32), t((7,), BF16)], norm=t((), F32), workspace=t((1 << 14,), U8))


CALLS = {
    "norm": _norm, "norm gradient": _norm_gradient,
    "gated": _of(layer.fp8_block_gated_gemm, {**GATED, **PLAIN}),
    "gated quantised": _of(layer.fp8_block_gated_gemm_quant, {**GATED, **QUANT}),
    "experts": _of(layer.fp8_block_grouped_gated_gemm, {**EXPERTS, **PLAIN}),
    "experts quantised": _of(layer.fp8_block_grouped_gated_gemm_quant, {**EXPERTS, **QUANT}),
    "gated gradient": _of(layer.fp8_gated_backward_quant, {"dh": ((128, 128), BF16), "gu": ((128, 256), BF16)}),
    "clip": _clip, "gradient norm": _grad_norm,
}


@pytest.mark.parametrize("other", ["cuda:1", "cpu"])
@pytest.mark.parametrize("name", CALLS)
def test_one_tensor_on_another_device(name, other, monkeypatch):
    monkeypatch.setattr(layer, "lib", lambda: pytest.fail("reached the library"))
    monkeypatch.setattr(layer, "_lib", None)
    monkeypatch.setattr(layer, "_current_gpu", lambda: 0, raising=False)
    with FakeTensorMode():
        def here(shape, dtype):
            return torch.empty(shape, dtype=dtype, device="cuda:0")

        def there(shape, dtype):
            return torch.empty(shape, dtype=dtype, device=other)

        fn, args = CALLS[name](here)
        _, moved = CALLS[name](there)
        for k, v in args.items():
            if isinstance(v, torch.Tensor):
                variants = [{**args, k: moved[k]}]
            elif isinstance(v, list):
                variants = [{**args, k: v[:i] + moved[k][i:i + 1] + v[i + 1:]} for i in range(len(v))]
            else:
                continue
            for kw in variants:
                with pytest.raises(ValueError, match="one GPU"):
                    fn(**kw)
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

    monkeypatch.setattr(layer, "_current_gpu", lambda: 0, raising=False)
    monkeypatch.setattr(torch.cuda, "device", Guard)
    for inner in ("_rows", "_gated_operands", "_gradients"):  # the checks that come next
        monkeypatch.setattr(layer, inner, reached)
    with FakeTensorMode():
        fn, args = CALLS[name](lambda shape, dtype: torch.empty(shape, dtype=dtype, device="cuda:1"))
        with pytest.raises(Reached):
            fn(**args)
    assert entered == [1]

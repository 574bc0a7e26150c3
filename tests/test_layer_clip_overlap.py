"""Clipping refuses lists whose outputs overlap: a tensor listed twice, a view inside another, an
output that is another tensor's gradient.  Refused on the host, so most of it needs no GPU."""

import ctypes
import random

import pytest
import torch

from fp8_fine_grained_amd import binding as fp8
from fp8_fine_grained_amd import layer

GOOD, NULL = ctypes.c_void_p(0x10000), ctypes.c_void_p(0)
F32, BF16 = fp8.F32, fp8.BF16


def _clip(grads, outs, counts, dtypes):
    n = len(grads)
    arr = lambda t, v: (t * n)(*v)  # noqa: E731
    L = layer.lib()
    return L.fp8fg_clip_grad_norm(arr(ctypes.c_void_p, grads), arr(ctypes.c_void_p, outs), arr(ctypes.c_int64, counts),
                                  arr(ctypes.c_int, dtypes), n, 1.0, GOOD, GOOD, L.fp8fg_grad_norm_workspace(n), NULL)


A, B, C = 0x100000, 0x200000, 0x300000


@pytest.mark.parametrize("grads,outs,counts,dtypes", [
    ([A, A], [A, A], [8, 8], [F32, F32]),                # listed twice
    ([A, B, A], [A, B, A], [8, 8, 8], [F32, F32, F32]),
    ([A, A + 16], [A, A + 16], [8, 8], [F32, F32]),      # a view that starts inside another
    ([A, A + 14], [A, A + 14], [8, 8], [BF16, BF16]),
    ([B, A], [B, A], [8, (B - A) // 4 + 1], [F32, F32]),
    ([A, B], [C, C], [8, 8], [F32, F32]),                # two outputs in one place
    ([A, B], [B, A], [8, 8], [F32, F32]),                # another tensor's gradient
    ([A, B], [C, A + 28], [8, 8], [F32, F32]),
    ([A], [A + 4], [8], [F32]),                          # its own in part
    ([A], [A - 28], [8], [F32]),
])
def test_overlaps_are_refused(grads, outs, counts, dtypes):
    assert _clip(grads, outs, counts, dtypes) == fp8.ERR_INVALID_ARG


def test_one_overlap_in_a_long_list_is_refused():
    rng = random.Random(0)
    for n in (63, 64, 65, 500):
        at = [A + 64 * i for i in range(n)]
        rng.shuffle(at)
        at[rng.randrange(n // 2)] = at[n - 1] + 60
        assert _clip(at, at, [16] * n, [F32] * n) == fp8.ERR_INVALID_ARG


@pytest.mark.gpu
def test_lists_that_touch_without_overlapping(gpu):
    """Neighbours in a flat buffer, empty tensors at one address, gradients read twice into separate outputs."""
    flat = torch.randn(1000, generator=torch.Generator().manual_seed(1)).to(gpu)
    want = flat * 0.5
    views = [flat[500:], flat[:3], flat[3:500], flat[3:3], flat[3:3]]
    norm = layer.grad_norm(views)
    layer.clip_grad_norm(views, float(norm) / 2)
    assert torch.allclose(flat, want, rtol=1e-6, atol=0)
    many = list(flat.clone().split(7))
    assert len(many) > 128
    layer.clip_grad_norm(many, 1e-3)
    a, outs = flat.clone(), [torch.empty(1000, device=gpu) for _ in range(2)]
    n2 = layer.clip_grad_norm([a, a], 1.0, out=outs)
    assert torch.equal(outs[0], outs[1]) and torch.isfinite(outs[0]).all()
    assert abs(float(n2) - 2 ** 0.5 * float(a.double().norm())) <= 1e-6 * float(n2)


@pytest.mark.gpu
def test_the_python_entry_point_refuses_too(gpu):
    t = torch.ones(300, device=gpu)
    with pytest.raises(fp8.Fp8fgError) as e:
        layer.clip_grad_norm([t, t], 1.0)
    assert e.value.status == fp8.ERR_INVALID_ARG
    with pytest.raises(fp8.Fp8fgError):
        layer.clip_grad_norm([t, t[:10]], 1.0)
    assert torch.all(t == 1)
    assert abs(float(layer.grad_norm([t, t])) - 600 ** 0.5) < 1e-4

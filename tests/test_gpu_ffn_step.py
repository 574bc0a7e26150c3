"""The feed-forward example: its gradients against 64-bit autograd of the same
sublayer, a few training steps, and single tokens against the training forward.

Bounds.  Every GEMM operand is rounded to E4M3 (relative error at most 2^-4,
uniform in between: 2^-4 / sqrt(3) = 0.036 rms at worst, 0.026 over a binade).  A
product's relative error is that of its operands added in squares; the forward
pass rounds n, w13, h and w2, and a gradient passes through at most four more
rounded operands and two of the forward's values: sqrt(8) * 0.026 = 0.073 at the
typical and sqrt(8) * 0.036 = 0.10 at the worst rounding.  0.12 is asked."""

import pytest
import torch

from examples.ffn_step import FeedForward, Server
from tests.gpu_util import say

pytestmark = pytest.mark.gpu


def _reference(ff, x, r):
    z = x.double() + r.double()
    n = z / torch.sqrt((z * z).mean(1, keepdim=True) + 1e-6) * ff["norm"]
    g, u = (n @ ff["w13"].t()).chunk(2, dim=1)
    return z + (g * torch.sigmoid(g) * u) @ ff["w2"].t()


def _rel(got, ref):
    return float((got.cpu().double() - ref).norm() / ref.norm())


@pytest.mark.parametrize("H,inner,T", [(256, 128, 128), (512, 640, 256)])
def test_gradients(gpu, H, inner, T):
    say(f"feed-forward gradients {H} {inner} {T}")
    ff = FeedForward(H, inner)
    gen = torch.Generator().manual_seed(3)
    x, r = (torch.randn((T, H), generator=gen).to(torch.bfloat16) for _ in range(2))
    dout = torch.randn((T, H), generator=gen).to(torch.bfloat16)
    p = {k: getattr(ff, k).cpu().double().requires_grad_() for k in ("norm", "w13", "w2")}
    xd = x.double().requires_grad_()
    ref = _reference(p, xd, r)
    ref.backward(dout.double())
    out, saved = ff.forward(x.to(gpu), r.to(gpu))
    dx, grads = ff.backward(dout.to(gpu), saved)
    z = x.double() + r.double()
    errs = {"out": _rel(out.cpu().double() - z, (ref - z).detach()), "dx": _rel(dx.cpu().double() - dout.double(),
                                                                             xd.grad - dout.double()),
            **{k: _rel(g, p[k].grad) for k, g in zip(("norm", "w13", "w2"), grads)}}
    say(str({k: round(v, 4) for k, v in errs.items()}))
    assert all(v <= 0.12 for v in errs.values()), errs


def test_training_reduces_the_loss(gpu):
    ff = FeedForward(256, 256)
    gen = torch.Generator(device="cuda").manual_seed(1)
    x, r = (torch.randn((256, 256), generator=gen, device="cuda").to(torch.bfloat16) for _ in range(2))
    target = (x + r).float() + 0.5 * torch.randn((256, 256), generator=gen, device="cuda")
    losses = [float(ff.step(x, r, target, 0.2)[0]) for _ in range(12)]
    say(f"losses {losses[0]:.3f} -> {losses[-1]:.3f}")
    assert losses[-1] < 0.9 * losses[0] and all(b < a * 1.02 for a, b in zip(losses, losses[1:]))


@pytest.mark.parametrize("tokens", [1, 5])
def test_serving_matches_the_training_forward(gpu, tokens):
    """Same weights, same sums; only h's rounding to bf16 before its quantisation differs
    (a code may move by one step: 0.03 of the feed-forward output is asked)."""
    ff = FeedForward(512, 256)
    server = Server(ff, tokens)
    gen = torch.Generator(device="cuda").manual_seed(2)
    for _ in range(3):
        x, r = (torch.randn((tokens, 512), generator=gen, device="cuda").to(torch.bfloat16) for _ in range(2))
        z = (x.float() + r.float()).double().cpu()
        got = server(x, r).double().cpu()
        out, _ = ff.forward(x, r)
        assert _rel(got - z, out.double().cpu() - z) <= 0.03

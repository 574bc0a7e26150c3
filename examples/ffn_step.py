"""A feed-forward sublayer in FP8, from the library's entry points: training steps and single tokens.

    python examples/ffn_step.py --steps 20            # train on a fixed synthetic regression
    python examples/ffn_step.py --serve               # one token at a time, timed in a HIP graph

Sublayer:  z = x + r,  out = z + W2 (silu(Wg n) * (Wu n)),  n = rmsnorm(z).  Weights are kept in fp32
and quantised 128x128 each step; activations and gradients are 1x128-quantised where a GEMM reads them.
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from fp8_fine_grained_amd import binding as fp8  # noqa: E402
from fp8_fine_grained_amd import layer  # noqa: E402


class FeedForward:
    """Weights (fp32): norm [H], w13 [2I, H] (gate rows, then up rows), w2 [H, I]."""

    def __init__(self, H, inner, seed=0, device="cuda"):
        gen = torch.Generator(device=device).manual_seed(seed)
        self.norm = torch.ones(H, device=device)
        self.w13 = torch.randn((2 * inner, H), generator=gen, device=device) * H ** -0.5
        self.w2 = torch.randn((H, inner), generator=gen, device=device) * inner ** -0.5

    def parameters(self):
        return [self.norm, self.w13, self.w2]

    def forward(self, x, r):
        """x, r bf16 [T, H] -> (out bf16 [T, H], what the backward pass reads)."""
        n = torch.empty_like(x)
        z, qn, sn, rstd = layer.fp8_add_rmsnorm_quant_1x128(x, self.norm, residual=r, y=n)
        q13, s13, q13t, s13t = fp8.fp8_quant_weight_128x128_dual(self.w13)
        q2, s2, q2t, s2t = fp8.fp8_quant_weight_128x128_dual(self.w2)
        qh, sh, gu = layer.fp8_block_gated_gemm_quant(qn, sn, q13, s13, save=True)
        out = z + fp8.fp8_block_gemm(qh, sh, q2, s2)
        return out, (n, z, rstd, gu, q13t, s13t, q2t, s2t)

    def backward(self, dout, saved):
        """dout bf16 [T, H] (T a multiple of 128) -> (dx, which is also dr, [dnorm, dw13, dw2])."""
        n, z, rstd, gu, q13t, s13t, q2t, s2t = saved
        q, s = fp8.fp8_quant_act_1x128(dout)
        qt, st = fp8.fp8_quant_act_1x128(dout.t())
        dh = fp8.fp8_block_gemm(q, s, q2t, s2t)
        q, s, dgut, dgut_s, ht, ht_s = layer.fp8_gated_backward_quant(dh, gu)
        dw2 = fp8.fp8_block_gemm(qt, st, ht, ht_s, b_scale_mode="row", accum="fp8", out_dtype=torch.float32)
        dn = fp8.fp8_block_gemm(q, s, q13t, s13t)
        qnt, snt = fp8.fp8_quant_act_1x128(n.t())
        dw13 = fp8.fp8_block_gemm(dgut, dgut_s, qnt, snt, b_scale_mode="row", accum="fp8", out_dtype=torch.float32)
        dx, dnorm = layer.fp8_rmsnorm_backward(dn, z, rstd, self.norm, dh=dout)
        return dx, [dnorm, dw13, dw2]

    def step(self, x, r, target, lr, max_norm=1.0):
        """One training step on the squared error; (loss, gradient norm before clipping), on the device."""
        out, saved = self.forward(x, r)
        diff = out.float() - target
        _, grads = self.backward((diff / x.shape[0]).to(torch.bfloat16), saved)
        norm = layer.clip_grad_norm(grads, max_norm)
        for w, g in zip(self.parameters(), grads):
            w.add_(g, alpha=-lr)
        return diff.square().sum(dim=1).mean() / 2, norm


class Server:
    """The sublayer for few tokens: weights quantised once, every buffer kept, one graph."""

    def __init__(self, ff, tokens=1):
        H, inner = ff.norm.numel(), ff.w2.shape[1]
        dev = ff.norm.device
        self.norm = ff.norm.to(torch.bfloat16)
        self.w13, self.w2 = fp8.fp8_quant_weight_128x128(ff.w13), fp8.fp8_quant_weight_128x128(ff.w2)
        self.x, self.r, self.z, self.y = (torch.zeros((tokens, H), dtype=torch.bfloat16, device=dev)
                                          for _ in range(4))
        self.n = (torch.empty((tokens, H), dtype=torch.uint8, device=dev),
                  torch.empty((tokens, H // 128), device=dev), torch.empty(tokens, device=dev))
        self.h = torch.empty((tokens, inner), dtype=torch.bfloat16, device=dev)
        self.qh = torch.empty((tokens, inner), dtype=torch.uint8, device=dev), torch.empty(
            (tokens, inner // 128), device=dev)
        self.run()
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self.run()

    def run(self):
        q, s, rstd = self.n
        layer.fp8_add_rmsnorm_quant_1x128(self.x, self.norm, residual=self.r, h=self.z, q=q, scales=s, rstd=rstd)
        layer.fp8_block_gated_gemm(q, s, *self.w13, h=self.h)
        fp8.fp8_quant_act_1x128(self.h, q=self.qh[0], scales=self.qh[1])
        fp8.fp8_block_gemm(*self.qh, *self.w2, y=self.y)
        self.y.add_(self.z)

    def __call__(self, x, r):
        self.x.copy_(x)
        self.r.copy_(r)
        self.graph.replay()
        return self.y


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--hidden", type=int, default=2048)
    ap.add_argument("--inner", type=int, default=2048)
    ap.add_argument("--tokens", type=int, default=1024, help="training tokens per step (a multiple of 128)")
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--lr", type=float, default=0.5)
    ap.add_argument("--serve", action="store_true")
    a = ap.parse_args()
    ff = FeedForward(a.hidden, a.inner)
    gen = torch.Generator(device="cuda").manual_seed(1)
    draw = lambda rows: torch.randn((rows, a.hidden), generator=gen, device="cuda").to(torch.bfloat16)  # noqa: E731
    if a.serve:
        server = Server(ff)
        x, r = draw(1), draw(1)
        server(x, r)
        beg, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        beg.record()
        for _ in range(200):
            server.graph.replay()
        end.record()
        torch.cuda.synchronize()
        print(f"one token through {a.hidden} x {a.inner}: {beg.elapsed_time(end) * 5:.1f} us")
        return
    x, r = draw(a.tokens), draw(a.tokens)
    target = (x + r).float() + 0.5 * draw(a.tokens).float()
    for k in range(a.steps):
        loss, norm = ff.step(x, r, target, a.lr)
        print(f"step {k}: loss {float(loss):.4f}, gradient norm {float(norm):.4f}", flush=True)


if __name__ == "__main__":
    main()

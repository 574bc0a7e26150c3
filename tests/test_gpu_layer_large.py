"""Layer operators on operands past 4 GiB: rows on both sides of the 2^32-byte and
2^31-element boundaries against 64-bit references of those rows alone."""

import pytest
import torch

from fp8_fine_grained_amd import binding, layer
from tests.gpu_util import say
from tests.layer_reference import U, check_close, check_quant
from tests.test_gpu_gated import _check_all, _reference

pytestmark = pytest.mark.gpu


def _codes(shape, seed):
    """Random finite E4M3 codes of both signs (exponents up to 2^1)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = torch.randint(0, 64, shape, generator=g, device="cuda", dtype=torch.uint8)
    return q | (torch.randint(0, 2, shape, generator=g, device="cuda", dtype=torch.uint8) << 7)


def test_norm_rows_past_4_gib(gpu):
    H = 7168
    M = (1 << 31) // H + 300  # bf16: the 2^32-byte boundary lies in row 2^31 / H
    say(f"norm {M}x{H}")
    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.empty((M, H), dtype=torch.bfloat16, device=gpu)
    for r in range(0, M, 65536):
        x[r:r + 65536] = torch.randn((min(65536, M - r), H), generator=g, device=gpu).to(torch.bfloat16)
    w = torch.rand(H, generator=g, device=gpu) + 0.5
    h, q, s, rstd = layer.fp8_add_rmsnorm_quant_1x128(x, w, residual=x)
    rows = [0, (1 << 30) // H, (1 << 31) // H - 1, (1 << 31) // H, (1 << 31) // H + 1, M - 1]
    z = 2 * x[rows].double().cpu()
    ref_rstd = 1 / torch.sqrt((z * z).mean(1) + 1e-6)
    y = z * ref_rstd[:, None] * w.double().cpu()
    check_close(h[rows], z, 0, "h")
    check_close(rstd[rows], ref_rstd, 32 * U, "rstd")
    check_quant(q[rows], s[rows], y, 40 * U)
    del h, q, s
    # (rows of the gradient: a column of ones in dy makes the others' dot easy to see)
    dx, _ = layer.fp8_rmsnorm_backward(x, x, rstd, w, need_dw=False)
    n = x[rows].double().cpu() * rstd[rows].double().cpu()[:, None]
    d = x[rows].double().cpu() * w.double().cpu()
    dot = (d * n).sum(1, keepdim=True)
    r = rstd[rows].double().cpu()[:, None]
    ref = r * (d - n * dot / H)
    floor = r * (8 * U * (d.abs() + (n * dot / H).abs()) + 64 * U * n.abs() * (d * n).abs().sum(1, keepdim=True) / H)
    check_close(dx[rows], ref, 2 * U, "dx", floor=floor)


def test_gated_tokens_past_4_gib(gpu):
    K, inner = 8192, 128
    M = (1 << 32) // K + 130
    say(f"gated {M}x{inner}x{K}")
    qa, sa = _codes((M, K), 1), torch.rand((M, K // 128), device=gpu) + 0.5
    qw, sw = _codes((2 * inner, K), 2), torch.rand((2 * inner // 128, K // 128), device=gpu) * 0.01
    h = layer.fp8_block_gated_gemm(qa, sa, qw, sw)
    rows = [0, (1 << 32) // K - 1, (1 << 32) // K, (1 << 32) // K + 1, M - 1]
    _check_all(_reference(qa[rows], sa[rows], qw, sw, "fp8"), "fp8", h[rows], what="tokens past 4 GiB")
    with pytest.raises(binding.Fp8fgError) as e:  # the grouped form's row offsets are 32-bit
        layer.fp8_block_grouped_gated_gemm(qa, sa, torch.tensor([0, M], dtype=torch.int32, device=gpu), qw[None],
                                           sw[None])
    assert e.value.status == binding.ERR_UNSUPPORTED


def test_experts_past_4_gib(gpu):
    K, inner = 4096, 1024
    G = (1 << 32) // (2 * inner * K) + 6
    say(f"gated experts {G} x {2 * inner}x{K}")
    qa, sa = _codes((40, K), 3), torch.rand((40, K // 128), device=gpu) + 0.5
    qw = _codes((G, 2 * inner, K), 4)
    sw = torch.rand((G, 2 * inner // 128, K // 128), device=gpu) * 0.01
    for per in (1, 20):  # the small workgroup shapes, and the tiles
        counts = torch.zeros(G, dtype=torch.int64)
        live = [0, G - 7, G - 6, G - 1]
        counts[live] = per
        off = torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)]).to(torch.int32).to(gpu)
        idx = (torch.arange(4 * per, dtype=torch.int32) * 7 % 40).to(gpu)
        h = layer.fp8_block_grouped_gated_gemm(qa, sa, off, qw, sw, row_index=idx)
        for k, e in enumerate(live):
            rows = idx[k * per:(k + 1) * per].long()
            _check_all(_reference(qa[rows], sa[rows], qw[e], sw[e], "fp8"), "fp8", h[k * per:(k + 1) * per],
                       what=f"expert {e}")


def test_gradient_of_the_activation_past_4_gib(gpu):
    M, inner = 1 << 17, 8448  # gu: 2^31 + 2^26 elements
    say(f"gated gradient {M}x{inner}")
    g = torch.Generator(device="cuda").manual_seed(5)
    dh = torch.empty((M, inner), dtype=torch.bfloat16, device=gpu)
    gu = torch.empty((M, 2 * inner), dtype=torch.bfloat16, device=gpu)
    for r in range(0, M, 16384):
        dh[r:r + 16384] = torch.randn((16384, inner), generator=g, device=gpu).to(torch.bfloat16)
        gu[r:r + 16384] = torch.randn((16384, 2 * inner), generator=g, device=gpu).to(torch.bfloat16)
    q, s, qt, st, qht, sht = layer.fp8_gated_backward_quant(dh, gu)
    from tests.test_gpu_gated import _grad_reference

    tokens = slice(M - 128, M)
    ref, floor, h = _grad_reference(dh[tokens].cpu(), gu[tokens].cpu())
    check_quant(q[tokens], s[tokens], ref, 4 * U, False, "rows", floor)
    cols = [0, inner - 1, inner, 2 * inner - 1]
    check_quant(qt[cols][:, tokens], st[cols][:, -1:], ref.t()[cols], 4 * U, False, "columns", floor.t()[cols])
    check_quant(qht[[0, inner - 1]][:, tokens], sht[[0, inner - 1]][:, -1:], h.t()[[0, inner - 1]], 20 * U, False,
                "h columns")


def test_clip_tensor_past_4_gib(gpu):
    n = (1 << 30) + 12345
    say(f"clip {n} fp32 values")
    x = torch.full((n,), 1e-3, device=gpu)
    x[-1] = 2.0
    out = [torch.empty_like(x), torch.empty(3, device=gpu)]
    norm = layer.clip_grad_norm([x, torch.ones(3, device=gpu)], 1.0, out=out)
    value = float(torch.tensor(1e-3).double())
    ref = ((n - 1) * value ** 2 + 4 + 3) ** 0.5
    assert abs(float(norm) - ref) <= 4 * U * ref
    at = [0, (1 << 29) - 1, 1 << 29, 1 << 30, n - 2, n - 1]
    check_close(out[0][at], x[at].double().cpu() / ref, 8 * U, "clipped")

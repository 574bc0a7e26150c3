"""The fused operators quantise by the very rule of fp8_quant_act_1x128: the same bits for the
same fp32 values, whatever the amax.

A gradient of the gated activation with g = 100 and u = 1 is dh itself (sigmoid(100) is 1 in fp32),
so dh goes into the fused quantiser unchanged and every mantissa of an amax can be given to it."""

import pytest
import torch

from fp8_fine_grained_amd import binding, layer
from tests.gpu_util import say
from tests.test_gpu_gated import _operands

pytestmark = pytest.mark.gpu


def _same(got, want, what):
    for a, b, name in zip(got, want, ("codes", "scales")):
        a, b = (t if t.dtype == torch.uint8 else t.view(torch.int32) for t in (a, b))
        assert torch.equal(a, b), f"{what}: {int((a != b).sum())} {name} differ"


def _through_the_gradient(dh, pow2=False):
    """Codes and scales of dh [M, 128] from the fused gradient: its gate half."""
    M = dh.shape[0]
    gu = torch.empty((M, 256), device=dh.device)
    gu[:, :128] = 100.0
    gu[:, 128:] = 1.0
    q, s = layer.fp8_gated_backward_quant(dh, gu, pow2=pow2, columns=False, h_columns=False)[:2]
    return q[:, :128].contiguous(), s[:, :1].contiguous()


@pytest.mark.parametrize("exponent", [-117, -100, -40, -1, 0, 8, 60, 127])
def test_every_mantissa_of_an_amax(gpu, exponent):
    """Exponents from the lowest of the rule's range (448 * 2^-126 lies in the binade of -118) to the highest."""
    say(f"scale rule 2^{exponent}")
    n = 1 << 23
    mantissa = torch.arange(n, device=gpu, dtype=torch.int32)
    amax = (mantissa | ((exponent + 127) << 23)).view(torch.float32)
    dh = torch.rand((n, 128), generator=torch.Generator(device=gpu).manual_seed(1), device=gpu)
    dh = (dh * 2 - 1) * amax[:, None]
    dh[torch.arange(n, device=gpu), torch.arange(n, device=gpu) % 128] = -amax
    for pow2 in (False, True):
        _same(_through_the_gradient(dh, pow2), binding.fp8_quant_act_1x128(dh, pow2=pow2), f"2^{exponent} pow2={pow2}")


def test_infinite_and_zero_groups(gpu):
    dh = torch.randn((3, 128), generator=torch.Generator().manual_seed(2)).to(gpu)
    dh[0, 9], dh[1, 50], dh[2] = float("inf"), -float("inf"), 0.0
    for pow2 in (False, True):
        _same(_through_the_gradient(dh, pow2), binding.fp8_quant_act_1x128(dh, pow2=pow2), f"pow2={pow2}")


@pytest.mark.parametrize("M,H", [(4096, 128), (300, 1152), (64, 7168)])
def test_norm(gpu, M, H):
    g = torch.Generator(device=gpu).manual_seed(3)
    x, w = torch.randn((M, H), generator=g, device=gpu) * 3, torch.rand(H, generator=g, device=gpu) + 0.5
    y = torch.empty_like(x)
    for pow2 in (False, True):
        _, q, s, _ = layer.fp8_add_rmsnorm_quant_1x128(x, w, y=y, pow2=pow2)
        _same((q, s), binding.fp8_quant_act_1x128(y, pow2=pow2), f"norm {M}x{H} pow2={pow2}")


@pytest.mark.parametrize("M,inner,K", [(1, 1024, 2048), (20, 2048, 512)])
def test_gated_product_of_few_rows(gpu, M, inner, K):
    """The small workgroup shapes leave h in the workspace in fp32 for the launch that quantises it."""
    for pow2 in (False, True):
        qa, sa, qw, sw = _operands(gpu, M, inner, K, False)
        nbytes = layer.lib().fp8_block_gated_gemm_quant_workspace(binding.ACCUM_FP8_MFMA, M, inner, K, 0)
        assert nbytes == 4 * M * inner, "not one of the small shapes"
        h = torch.empty((M, inner), device=gpu)
        got = layer.fp8_block_gated_gemm_quant(qa, sa, qw, sw, pow2=pow2, workspace=h)
        _same(got, binding.fp8_quant_act_1x128(h, pow2=pow2), f"gated {M}x{inner}x{K} pow2={pow2}")


@pytest.mark.parametrize("accum", ["fp8", "exact", "scaled"])
def test_infinite_outputs_do_not_depend_on_the_workgroup_shape(gpu, accum):
    """h of the first row overflows fp32: its groups have the same codes and scales from the kernel
    that holds whole groups and from the one that leaves them to a second launch."""
    M, inner, K = 3, 1024, 2048
    g = torch.Generator().manual_seed(4)
    a = torch.full((M, K), 0x38, dtype=torch.uint8)  # 1.0
    w = torch.where(torch.rand((2 * inner, K), generator=g) < 0.5, 0x38, 0xB8).to(torch.uint8)  # +-1.0
    sa = torch.ones((M, K // 128))
    sa[0] = 2.0 ** 32
    sw = torch.full((2 * inner // 128, K // 128), 2.0 ** 34)
    ops = [t.to(gpu) for t in (a, sa, w, sw)]
    mode = binding._accum_code(accum, torch.bfloat16)
    assert layer.lib().fp8_block_gated_gemm_quant_workspace(mode, M, inner, K, 0) > 0
    none = torch.empty(0, dtype=torch.uint8, device=gpu)
    for pow2 in (False, True):
        small = layer.fp8_block_gated_gemm_quant(*ops, accum=accum, pow2=pow2)
        whole = layer.fp8_block_gated_gemm_quant(*ops, accum=accum, pow2=pow2, workspace=none)
        assert torch.isinf(whole[1][0]).all() or pow2
        _same(small, whole, f"{accum} pow2={pow2}")

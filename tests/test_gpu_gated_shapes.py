"""Every workgroup shape of the gated products in every form: sums, output types, kept gate and
up values, quantised outputs through the workspace and without it.  (Another test asks the
library's rule that these sizes take them all.)"""

import pytest
import torch

from fp8_fine_grained_amd import layer
from tests.gated_sizes import DENSE, EXPERTS
from tests.gpu_util import say
from tests.test_gpu_gated import _check_all, _operands, _reference, _segments

pytestmark = pytest.mark.gpu


def _rows(M):
    """All rows of few, else those around the edges of the shapes' tiles."""
    if M <= 64:
        return list(range(M))
    near = {r + d for r in (0, 16, 32, 64, 128, 256, 512, 1024, M) for d in (-2, -1, 0, 1)}
    return sorted({r for r in near if 0 <= r < M} | set(range(0, M, 37)))


@pytest.mark.parametrize("accum", ["fp8", "exact", "scaled"])
@pytest.mark.parametrize("M,inner,K", DENSE)
def test_dense(gpu, M, inner, K, accum):
    say(f"gated shapes {M}x{inner}x{K} {accum}")
    ops = _operands(gpu, M, inner, K, accum == "scaled")
    at = _rows(M)
    ref = _reference(ops[0][at], ops[1][at], *ops[2:], accum)
    what = f"{M}x{inner}x{K} {accum}"
    h, gu = layer.fp8_block_gated_gemm(*ops, accum=accum, save=True)
    _check_all(ref, accum, h[at], gu[at], what=what + " bf16")
    assert torch.equal(layer.fp8_block_gated_gemm(*ops, accum=accum), h)
    h, gu = layer.fp8_block_gated_gemm(*ops, accum=accum, out_dtype=torch.float32, save=True)
    _check_all(ref, accum, h[at], gu[at], what=what + " f32")
    none = torch.empty(0, dtype=torch.uint8, device=gpu)
    for pow2 in (False, True):
        for ws in (None, none):
            q, s, gu = layer.fp8_block_gated_gemm_quant(*ops, accum=accum, pow2=pow2, save=True, workspace=ws)
            _check_all(ref, accum, gu=gu[at], quant=(q[at], s[at]), pow2=pow2, what=f"{what} quantised {ws is None}")


@pytest.mark.parametrize("accum", ["fp8", "exact", "scaled"])
@pytest.mark.parametrize("counts,inner,K", EXPERTS)
def test_experts(gpu, counts, inner, K, accum):
    G, R, tokens = len(counts), sum(counts), 50
    say(f"gated shapes, experts {counts} {inner}x{K} {accum}")
    qa, sa, qw, sw = _operands(gpu, tokens, inner, K, accum == "scaled", G=G)
    off = _segments(counts).to(gpu)
    idx = torch.randint(0, tokens, (R,), generator=torch.Generator().manual_seed(R), dtype=torch.int32).to(gpu)
    call = dict(row_index=idx, accum=accum)
    h, gu = layer.fp8_block_grouped_gated_gemm(qa, sa, off, qw, sw, save=True, **call)
    f, gf = layer.fp8_block_grouped_gated_gemm(qa, sa, off, qw, sw, save=True, out_dtype=torch.float32, **call)
    none = torch.empty(0, dtype=torch.uint8, device=gpu)
    quant = {(pow2, ws is None): layer.fp8_block_grouped_gated_gemm_quant(qa, sa, off, qw, sw, pow2=pow2, save=True,
                                                                          workspace=ws, **call)
             for pow2 in (False, True) for ws in (None, none)}
    li = idx.long()
    assert torch.equal(layer.fp8_block_grouped_gated_gemm(qa[li], sa[li], off, qw, sw, accum=accum), h)
    for e in range(G):
        lo, hi = int(off[e]), int(off[e + 1])
        if lo == hi:
            continue
        at = torch.tensor(_rows(hi - lo), device=gpu) + lo
        ref = _reference(qa[li[at]], sa[li[at]], qw[e], sw[e], accum)
        _check_all(ref, accum, h[at], gu[at], what=f"expert {e} bf16")
        _check_all(ref, accum, f[at], gf[at], what=f"expert {e} f32")
        for (pow2, ws), (q, s, gq) in quant.items():
            _check_all(ref, accum, gu=gq[at], quant=(q[at], s[at]), pow2=pow2, what=f"expert {e} quantised {ws}")

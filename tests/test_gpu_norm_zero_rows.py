"""Rows of zeros (padding) and rows whose squares vanish in fp32, with eps == 0: they have no
direction, so the norm of such a row is defined as zero (rstd 0), forward and backward."""

import pytest
import torch

from fp8_fine_grained_amd import layer
from tests.layer_reference import U, check_close, check_quant
from tests.test_gpu_norm import REL_RSTD, REL_Y, _check_backward, _inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,H", [(4, 128), (9, 640), (5, 7168), (6, 16512)])
def test_zero_and_vanishing_rows_without_eps(gpu, M, H, dtype):
    x, r, w = _inputs(M, H, dtype)
    none, tiny = 1, 3
    for t in (x, r):
        t[none] = 0
        t[tiny] = 1e-25
    dead = [none, tiny]
    live = [m for m in range(M) if m not in dead]
    for residual in (None, r):
        z = x.double() + (residual.double() if residual is not None else 0)
        for pow2 in (False, True):
            yo = torch.empty((M, H), dtype=dtype, device=gpu)
            h, q, s, rstd = layer.fp8_add_rmsnorm_quant_1x128(
                x.to(gpu), w.to(gpu), residual=None if residual is None else residual.to(gpu), eps=0.0, pow2=pow2, y=yo)
            assert torch.all(rstd[dead] == 0) and torch.all(yo[dead] == 0)
            assert torch.all(q[dead] & 0x7F == 0) and torch.all(s[dead] == 0)
            ref = 1 / torch.sqrt((z[live] ** 2).mean(1))
            check_close(rstd[live], ref, REL_RSTD, "rstd")
            check_quant(q[live], s[live], z[live] * ref[:, None] * w.double(), REL_Y, pow2)
            check_close(h, z, 0, "h", floor=U * float(z.abs().max()))
        # the gradient of such a row is what arrives along the residual stream, and dw is that of the others
        dy = (r.float() * 0.5 + 1e-3).to(dtype)
        for dh in (None, r):
            args = [t.to(gpu) for t in (dy, h.cpu(), rstd.cpu(), w)]
            dx, dw = layer.fp8_rmsnorm_backward(*args, dh=None if dh is None else dh.to(gpu))
            assert torch.equal(dx[dead].cpu(), torch.zeros((2, H), dtype=dtype) if dh is None else dh[dead])
            _check_backward(dy[live], h.cpu()[live], rstd.cpu()[live], w, None if dh is None else dh[live], dx[live],
                            dw, "others")

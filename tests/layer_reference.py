"""64-bit references and bounds for the layer operators (norm, gated, clipping).

All in torch float64 on the CPU, from the operators' formulas.  The bounds count
fp32 roundings: ``U`` is the unit roundoff of fp32, ``UB`` that of bf16.
"""

import torch

U = 2.0 ** -24
UB = 2.0 ** -8  # half an ulp of bf16, relative to the value's power of two
E4M3_MAX = 448.0


def e4m3_values(q):
    return q.cpu().view(torch.float8_e4m3fn).double()


def check_quant(q, scales, ref, rel, pow2=False, what="", floor=None):
    """Codes [M, K] and scales [M, K/128] against the 64-bit values ``ref`` that
    the kernel holds in fp32 to within ``rel`` of each value plus ``floor``
    [M, K] (absolute) before quantising.

    Scales: amax/448 to within rel, floor and two roundings, or the power of two
    whose range holds the amax.  Codes: the value times the kernel's own scale
    is within half an E4M3 step of ref, plus the error of the value and two
    roundings of the scaled value."""
    M, K = ref.shape
    q, s = e4m3_values(q).view(M, K // 128, 128), scales.cpu().double()
    r = ref.cpu().double().view(M, K // 128, 128)
    amax = r.abs().amax(dim=2)
    fl = torch.zeros_like(r) if floor is None else floor.cpu().double().view(M, K // 128, 128)
    err = rel * amax + fl.amax(dim=2)
    if pow2:
        nz = s > 0
        m, _ = torch.frexp(s[nz])
        assert torch.all(m == 0.5), f"{what}: a scale is not a power of two"
        assert torch.all(amax[nz] <= E4M3_MAX * s[nz] + err[nz]), f"{what}: scale too small"
        assert torch.all(amax[nz] + err[nz] > E4M3_MAX / 2 * s[nz]), f"{what}: scale too large"
        assert torch.all(amax[~nz] <= err[~nz]), f"{what}: zero scale for a nonzero group"
    else:
        assert torch.all((s - amax / E4M3_MAX).abs() <= err / E4M3_MAX + 2 * U * s), f"{what}: scales"
    safe = torch.where(s > 0, s, torch.ones_like(s))[:, :, None]
    v = r / safe
    off = v.abs() * (rel + 4 * U) + fl / safe  # how far the scaled value may be from v
    # the step of the largest value it may be
    _, e = torch.frexp(v.abs() + off)
    step = torch.exp2((e - 1).clamp(min=-6).double() - 3)
    tol = step / 2 + off
    bad = ~((q - v).abs() <= tol) & (s > 0)[:, :, None]  # (a NaN is within no bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} codes off, first {bad.nonzero()[:3].tolist()}"
    assert torch.all(q[s == 0] == 0), f"{what}: codes of a zero group"


def check_close(got, ref, rel, what, dtype=None, floor=0.0):
    """|got - ref| <= rel |ref| + floor, plus the rounding to the output type."""
    g, r = got.cpu().double(), ref.cpu().double()
    round_to = UB if (dtype or got.dtype) == torch.bfloat16 else U
    tol = (rel + round_to) * r.abs() + floor + 2.0 ** -133
    bad = ~((g - r).abs() <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} values off, worst "
                           f"{float(((g - r).abs() / tol).nan_to_num(1e9).max()):.2f} of the bound")


def silu(g):
    return g * torch.sigmoid(g)


def gated_bound(g, u, dg, du, rel):
    """Bound of |h - silu(g) u| when g and u are off by at most dg and du and the
    activation's own arithmetic is off by rel: |silu'| <= 1.1 everywhere."""
    return 1.1 * u.abs() * dg + silu(g).abs() * du + 1.1 * dg * du + rel * (silu(g) * u).abs()

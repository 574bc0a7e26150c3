"""64-bit references of the expert layer's operators, in torch float64 (or integers) on the CPU, from the
operators' formulas."""

import torch

from tests.layer_reference import U

E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
OUT = -float("inf")
NAN_RANK = -1e300  # what is not a number: below all fp32 numbers, above what is out


def scores(z, score):
    """s [T, E] in 64 bits; a logit of -infinity has score 0."""
    z = z.double()
    if score == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-z))
    m = z.nan_to_num(nan=OUT, posinf=float("inf"), neginf=OUT).amax(dim=1, keepdim=True)
    e = torch.where(z == OUT, 0.0, torch.exp(z - m))
    return torch.where(e == 0, 0.0, e / e.sum(dim=1, keepdim=True))


def shares(z, at, there, score):
    """s / sum of s over the chosen experts [T, k], from logarithms: the scores may be too small for any type."""
    q = z.double().gather(1, at)
    q = torch.where(there, q, OUT)
    f = torch.nn.functional.logsigmoid(q) if score == "sigmoid" else q
    m = f.nan_to_num(nan=OUT, posinf=float("inf"), neginf=OUT).amax(dim=1, keepdim=True)
    f = torch.where(f == OUT, 0.0, torch.exp(f - m))
    return torch.where(f == 0, 0.0, f / f.sum(dim=1, keepdim=True))


def rel_scores(z, score):
    """Relative error of an fp32 score [T, 1], counted in roundings: the exponential (2), its argument (for softmax
    the rounded difference from the largest logit, off by up to U times itself), the sum (16 in a lane, 6 over
    lanes), the division."""
    if score == "sigmoid":
        return torch.full((z.shape[0], 1), 6 * U, dtype=torch.float64)
    f = z.double().nan_to_num(nan=0.0, posinf=0.0, neginf=0.0)
    return (f.amax(dim=1, keepdim=True) - f.amin(dim=1, keepdim=True) + 30) * U


def _best(v, n):
    """Indices of the n largest of each row, descending, ties to the lowest index."""
    return torch.sort(v, dim=1, descending=True, stable=True)[1][:, :n]


def route(z, k, bias=None, mask=None, score="sigmoid", groups=1, groups_kept=1, group_terms=2, renormalise=True,
          scale=1.0):
    """(experts int32 [T, k], weights float64 [T, k], scores float64 [T, E])."""
    z = z.cpu()
    bias = None if bias is None else bias.cpu()
    T, E = z.shape
    s = scores(z, score)
    b = torch.zeros(E, dtype=torch.float64) if bias is None else bias.double()
    c = s + b
    gone = (z.double() == OUT) | (b == OUT)

    def rank(v):
        return torch.where(gone, OUT, torch.where(v.isnan(), NAN_RANK, v))

    key = rank(z.double() if bias is None else c)
    if groups_kept < groups:
        v = (rank(c) if bias is not None or group_terms == 2 else key).view(T, groups, -1)
        top = torch.sort(v, dim=2, descending=True)[0][:, :, :group_terms]
        value = torch.where((top == OUT).any(dim=2), OUT, top.sum(dim=2))
        keep = torch.zeros((T, groups), dtype=torch.bool).scatter(1, _best(value, groups_kept), True) & (value != OUT)
        key = torch.where(keep.repeat_interleave(E // groups, dim=1), key, OUT)
    experts = _best(key, k)
    there = key.gather(1, experts) != OUT
    if mask is not None:
        there &= (mask.cpu() != 0)[:, None]
    w = shares(z, experts, there, score) if renormalise else torch.where(there, s.gather(1, experts), 0.0)
    return torch.where(there, experts, -1).int(), w * scale, s


def route_backward(dw, experts, z, score, renormalise, scale, ds=None):
    """(dz, the sum of the magnitudes that its roundings are relative to), float64 [T, E]."""
    dw, z, experts = dw.cpu().double(), z.cpu(), experts.cpu().long()
    s = scores(z, score)
    E = z.shape[1]
    there = (experts >= 0) & (experts < E)
    at = experts.clamp(0, E - 1)
    q = torch.where(there, s.gather(1, at), 0.0)
    g = torch.where(there, dw * scale, 0.0)
    if renormalise:
        p = shares(z, at, there, score)
        t = p * (g - (g * p).sum(dim=1, keepdim=True))
        ta = p * (g.abs() + (g * p).abs().sum(dim=1, keepdim=True))
    else:
        t, ta = q * g, (q * g).abs()
    d, da = torch.zeros_like(s), torch.zeros_like(s)
    d.scatter_add_(1, at, t)
    da.scatter_add_(1, at, ta)
    if ds is not None:
        d += ds.cpu().double() * s
        da += (ds.cpu().double() * s).abs()
    if score == "sigmoid":
        dz, size = d * (1 - s), da * (1 - s) + d.abs() * s
    else:
        dz = d - s * d.sum(dim=1, keepdim=True)
        size = da + s * da.sum(dim=1, keepdim=True)
    gone = z.double() == OUT
    return torch.where(gone, 0.0, dz), torch.where(gone, 0.0, size)


def segments(experts, G, first=0):
    """(offsets, row_index, positions) as lists, by going through the entries."""
    e = experts.cpu().tolist()
    T, k = experts.shape
    rows = [[] for _ in range(G)]
    for t in range(T):
        for j in range(k):
            if first <= e[t][j] < first + G:
                rows[e[t][j] - first].append((t, j))
    offsets, row_index, positions = [0], [], [[-1] * k for _ in range(T)]
    for r in rows:
        for t, j in r:
            positions[t][j] = len(row_index)
            row_index.append(t)
        offsets.append(len(row_index))
    return offsets, row_index + [0] * (T * k - len(row_index)), positions


def combine(rows, positions, weights=None, base=None):
    """(y, sum of magnitudes), float64 [T, H]."""
    rows, positions = rows.cpu().double(), positions.cpu().long()
    T, k = positions.shape
    y = torch.zeros((T, rows.shape[1]), dtype=torch.float64) if base is None else base.cpu().double().clone()
    size = y.abs()
    for j in range(k):
        p = positions[:, j]
        t = ((p >= 0) & (p < rows.shape[0])).nonzero().flatten()
        v = rows[p[t]] * (1.0 if weights is None else weights.cpu().double()[t, j, None])
        y[t] += v
        size[t] += v.abs()
    return y, size


def combine_backward(dy, positions, weights, rows, R):
    """(drows float64 [R, H] (NaN where nothing is written), dweights [T, k], their sums of magnitudes)."""
    dy, positions = dy.cpu().double(), positions.cpu().long()
    T, k = positions.shape
    d = torch.full((R, dy.shape[1]), float("nan"), dtype=torch.float64)
    dw, size = torch.zeros((T, k), dtype=torch.float64), torch.zeros((T, k), dtype=torch.float64)
    for j in range(k):
        p = positions[:, j]
        t = ((p >= 0) & (p < R)).nonzero().flatten()
        d[p[t]] = dy[t] * (1.0 if weights is None else weights.cpu().double()[t, j, None])
        if rows is not None:
            v = dy[t] * rows.cpu().double()[p[t]]
            dw[t, j], size[t, j] = v.sum(dim=1), v.abs().sum(dim=1)
    return d, dw, size


def fp4_quant(w):
    """(codes uint8 [N, K/2], scales uint8 [N, K/32]) by the rule, from exact 64-bit arithmetic."""
    N, K = w.shape
    g = w.cpu().double().view(N, K // 32, 32)
    m, e = torch.frexp(g.abs().amax(dim=2))  # 6 2^e: (0.75, e + 3)
    e = (e - 3 + (m > 0.75).int()).clamp(min=-126)
    e = torch.where(m == 0, torch.full_like(e, -126), e)
    v = (g.abs() * torch.exp2(-e.double())[:, :, None]).flatten()
    lo = (torch.searchsorted(E2M1, v, right=True) - 1).clamp(max=6)
    below, above = v - E2M1[lo], E2M1[lo + 1] - v
    up = (above < below) | ((above == below) & (lo % 2 == 1))  # ties to the even code
    code = (lo + up.long()) | (torch.signbit(g.flatten()).long() << 3)
    code = code.view(N, K // 2, 2)
    return (code[:, :, 0] | (code[:, :, 1] << 4)).to(torch.uint8), (e + 127).to(torch.uint8)


def fp4_values(q, scales):
    """Weights [.., N, K] in float64."""
    q, scales = q.cpu().long(), scales.cpu()
    code = torch.stack([q & 15, q >> 4], dim=-1).flatten(-2)
    v = torch.where(code >= 8, -E2M1[code & 7], E2M1[code & 7])
    return v * torch.exp2(scales.double() - 127).repeat_interleave(32, dim=-1)


def x_values(x, sx=None):
    x = x.cpu()
    if sx is None:
        return x.double()
    return x.view(torch.float8_e4m3fn).double() * sx.cpu().double().repeat_interleave(128, dim=1)


def fp4_product(x, w):
    """(x w^T, the sum of the magnitudes of its products), float64."""
    return x @ w.t(), x.abs() @ w.t().abs()

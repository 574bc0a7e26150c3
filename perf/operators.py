"""Cases of the operators around the FP8 GEMM: what is measured, in plain torch and in the library.

Three operators, each with the shapes a feed-forward sublayer of an FP8 training step meets:

* ``norm``  residual addition, root-mean-square norm and 1x128 E4M3 quantisation in one pass, and the
            norm's gradient (``norm_grad``);
* ``gated`` the gated feed-forward pair of block-scaled FP8 products with its activation, dense, for a
            single token, quantised, and over expert segments (``experts``), and its gradient, left
            1x128-quantised along both axes (``gated_grad``);
* ``clip``  the global norm over many gradients and their clipping.

With ``own`` false, ``run`` computes them by elementary torch operations in 32 bits; with ``own`` true it
calls the library.  E4M3 codes are returned as torch.float8_e4m3fn, the values they stand for.
"""

import math

import torch

own = False

E4M3_MAX = 448.0
EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one token entering the feed-forward sublayer while serving: latency
        {"name": "norm token", "op": "norm", "M": 1, "H": 7168, "dtype": "bf16", "residual": True, "pow2": False},
        # the dense projection's tokens, as a training step norms them
        {"name": "norm step", "op": "norm", "M": 4096, "H": 7168, "dtype": "bf16", "residual": True, "pow2": False},
        # an odd number of fp32 rows without a residual, power-of-two scales
        {"name": "norm odd f32 pow2", "op": "norm", "M": 1037, "H": 2176, "dtype": "f32", "residual": False,
         "pow2": True},
        # the same tokens in the backward pass, with the gradient that arrives along the residual stream
        {"name": "norm gradient", "op": "norm_grad", "M": 4096, "H": 7168, "dtype": "bf16", "residual": True},
        # few fp32 rows of a narrow model
        {"name": "norm gradient small f32", "op": "norm_grad", "M": 333, "H": 640, "dtype": "f32",
         "residual": False},
        # one token through an expert-sized pair of projections while serving
        {"name": "gated token", "op": "gated", "M": 1, "I": 2048, "K": 7168, "form": "bf16"},
        # a ragged batch, exact products, output left quantised for the down projection
        {"name": "gated ragged quantised", "op": "gated", "M": 777, "I": 1152, "K": 2304, "form": "quant"},
        # the dense layer's pair of projections in a training step, keeping what its gradient reads
        {"name": "gated step", "op": "gated", "M": 4096, "I": 18432, "K": 7168, "form": "saved"},
        # one GPU's share of the expert layer: 32 of 256 experts, some of them empty, rows read by index
        {"name": "gated experts", "op": "experts", "T": 8192, "rows": 8192, "G": 32, "empty": 3, "I": 2048,
         "K": 7168},
        # the gradient of that share's activation, for both products of the backward pass
        {"name": "gated gradient", "op": "gated_grad", "M": 8192, "I": 2048, "dtype": "bf16", "pow2": False},
        # a handful of small gradients of both types and of odd lengths: latency
        {"name": "clip small", "op": "clip", "tensors": 14, "numel": 90001, "share": 0.3, "ratio": 3.0},
        # the weight gradients of the dense feed-forward layer, most of them fp32
        {"name": "clip layer", "op": "clip", "tensors": 24, "numel": 396361728, "share": 0.1, "ratio": 20.0},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _log_128(rng, lo, hi):
    """A multiple of 128 in [lo, hi]."""
    return 128 * _log_int(rng, lo // 128, hi // 128)


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "gated", "gated", "experts", "gated_grad", "clip"])
    if op in ("norm", "norm_grad"):
        H = _log_128(rng, 128, 18432)
        M = _log_int(rng, 1, min(16384, (1 << 27) // H))
        case = {"op": op, "M": M, "H": H, "dtype": rng.choice(["bf16", "f32"]), "residual": rng.random() < 0.7}
        if op == "norm":
            case["pow2"] = rng.random() < 0.4
        return case
    if op == "gated":
        K = _log_128(rng, 256, 16384)
        inner = _log_128(rng, 128, min(18432, 18432 * 7168 // K // 128 * 128))
        M = _log_int(rng, 1, 4096)
        return {"op": op, "M": M, "I": inner, "K": K, "form": rng.choice(["bf16", "saved", "quant"])}
    if op == "experts":
        G = _log_int(rng, 2, 64)
        K = _log_128(rng, 512, 7168)
        inner = _log_128(rng, 128, max(128, min(2048, 32 * 2048 * 7168 // (G * K) // 128 * 128)))
        T = _log_int(rng, 1, 4096)
        return {"op": op, "T": T, "rows": T * rng.randint(1, 2), "G": G, "empty": rng.randint(0, G // 2), "I": inner,
                "K": K}
    if op == "gated_grad":
        inner = _log_128(rng, 128, 18432)
        M = _log_int(rng, 1, min(8192, (1 << 25) // inner))
        if M >= 128 and rng.random() < 0.7:
            M = M // 128 * 128
        return {"op": op, "M": M, "I": inner, "dtype": rng.choice(["bf16", "f32"]), "pow2": rng.random() < 0.4}
    return {"op": op, "tensors": rng.randint(1, 60), "numel": _log_int(rng, 1000, 1 << 27),
            "share": rng.choice([0.0, 0.3, 1.0]), "ratio": rng.choice([0.5, 2.0, 10.0])}


# ------------------------------------------------------------------ inputs
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(gen, shape, std=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=gen, device="cuda") * std).to(dtype)


def _outliers(gen, x, share=0.001, factor=100.0):
    """Some entries enlarged, as the channels of a residual stream have them."""
    return torch.where(torch.rand(x.shape, generator=gen, device="cuda") < share, x * factor, x)


def _quant_rows(x, pow2=False):
    """1x128 codes (float8) and scales of x [M, K] in 32 bits."""
    g = x.float().reshape(x.shape[0], -1, 128)
    s = _scale(g.abs().amax(dim=2), pow2)
    inv = torch.where(s == 0, torch.zeros_like(s), 1.0 / s)
    return (g * inv[:, :, None]).to(torch.float8_e4m3fn).reshape(x.shape), s


def _scale(amax, pow2):
    if not pow2:
        return amax / E4M3_MAX
    m, e = torch.frexp(amax)  # amax = m 2^e, m in [1/2, 1); 448 = 0.875 * 2^9
    e = e - 9 + (m > 0.875).to(e.dtype)
    return torch.where(amax == 0, torch.zeros_like(amax), torch.ldexp(torch.ones_like(amax), e))


def _quant_blocks(w):
    """128x128 codes (uint8) and scales of w [N, K]."""
    N, K = w.shape
    g = w.float().reshape(N // 128, 128, K // 128, 128)
    s = g.abs().amax(dim=(1, 3)) / E4M3_MAX
    q = (g / s[:, None, :, None]).to(torch.float8_e4m3fn).reshape(N, K)
    return q.view(torch.uint8), s


def _quant_weights(gen, rows, K):
    """Codes and scales of a weight [rows, K] ~ N(0, 0.02), drawn a few blocks of rows at a time."""
    q = torch.empty((rows, K), dtype=torch.uint8, device="cuda")
    s = torch.empty((rows // 128, K // 128), dtype=torch.float32, device="cuda")
    step = max(128, (1 << 26) // K // 128 * 128)
    for r in range(0, rows, step):
        n = min(step, rows - r)
        q[r:r + n], s[r // 128:(r + n) // 128] = _quant_blocks(_normal(gen, (n, K), 0.02))
    return q, s


def _tensors(case):
    """(length, type) of each gradient: one or two hold most of the values, the others have odd lengths."""
    n, total = case["tensors"], case["numel"]
    big = [total * 2 // 3, total // 4][: min(2, n - 1)] if n > 1 else [total]
    gen = torch.Generator().manual_seed(n + total)
    cuts, narrow = torch.rand(n - len(big), generator=gen), torch.rand(n, generator=gen) < case["share"]
    sizes = big + [int((total - sum(big)) * float(c) / n) | 1 for c in cuts]
    return [(k, torch.bfloat16 if b else torch.float32) for k, b in zip(sizes, narrow.tolist())]


def prepare(case, seed):
    gen = _generator(seed)
    op, s = case["op"], {"case": case}
    if op == "norm":
        dt = DTYPES[case["dtype"]]
        shape = (case["M"], case["H"])
        s["x"] = _outliers(gen, _normal(gen, shape)).to(dt)
        s["r"] = _normal(gen, shape, 2.0, dt) if case["residual"] else None
        s["w"] = (1.0 + _normal(gen, (case["H"],), 0.1)).to(dt)
    elif op == "norm_grad":
        dt = DTYPES[case["dtype"]]
        shape = (case["M"], case["H"])
        s["dy"] = _normal(gen, shape, 1e-3, dt)
        s["h"] = _outliers(gen, _normal(gen, shape, 2.0)).to(dt)
        s["rstd"] = (s["h"].float().square().mean(dim=1) + EPS).sqrt().reciprocal()
        s["w"] = (1.0 + _normal(gen, (case["H"],), 0.1)).to(dt)
        s["dh"] = _normal(gen, shape, 1e-3, dt) if case["residual"] else None
    elif op in ("gated", "experts"):
        rows = case["M"] if op == "gated" else case["T"]
        a, s["sa"] = _quant_rows(_outliers(gen, _normal(gen, (rows, case["K"]))))
        s["a"] = a.view(torch.uint8)
        G = 1 if op == "gated" else case["G"]
        w, sw = _quant_weights(gen, G * 2 * case["I"], case["K"])
        if op == "gated":
            s["w"], s["sw"] = w, sw
        else:
            s["w"], s["sw"] = w.view(G, 2 * case["I"], case["K"]), sw.view(G, 2 * case["I"] // 128, -1)
            live = torch.randperm(G, generator=gen, device="cuda")[: G - case["empty"]]
            pick = torch.randint(0, len(live), (case["rows"],), generator=gen, device="cuda")
            counts = torch.bincount(live[pick], minlength=G)
            s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
            s["rows"] = torch.randint(0, case["T"], (case["rows"],), generator=gen, device="cuda").to(torch.int32)
            s["most"] = int(counts.max())
    elif op == "gated_grad":
        dt = DTYPES[case["dtype"]]
        s["dh"] = _normal(gen, (case["M"], case["I"]), 1e-3, dt)
        s["gu"] = _normal(gen, (case["M"], 2 * case["I"]), 1.7, dt)
    else:
        std = case["ratio"] / math.sqrt(sum(k for k, _ in _tensors(case)))  # the norm is about `ratio`, the limit 1
        s["grads"] = [_normal(gen, (k,), std, dt) for k, dt in _tensors(case)]
        s["out"] = [torch.empty_like(g) for g in s["grads"]]
    return s


# ------------------------------------------------------------------ plain forms (32 bits)
def _dequant_rows(q, s):
    return q.view(torch.float8_e4m3fn).float() * s.repeat_interleave(128, dim=1)


def _dequant_blocks(q, s):
    return q.view(torch.float8_e4m3fn).float() * s.repeat_interleave(128, dim=-2).repeat_interleave(128, dim=-1)


def _norm(s):
    case, z = s["case"], s["x"].float()
    if s["r"] is not None:
        z = z + s["r"].float()
    rstd = (z.square().mean(dim=1) + EPS).sqrt().reciprocal()
    q, scales = _quant_rows(z * rstd[:, None] * s["w"].float(), case["pow2"])
    return {"h": z.to(s["x"].dtype), "q": q, "scales": scales, "rstd": rstd}


def _norm_grad(s):
    dy, n = s["dy"].float(), s["h"].float() * s["rstd"][:, None]
    d = dy * s["w"].float()
    dx = s["rstd"][:, None] * (d - n * (d * n).mean(dim=1, keepdim=True))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return {"dx": dx.to(s["dy"].dtype), "dw": (dy * n).sum(dim=0)}


def _activate(gu):
    g, u = gu.chunk(2, dim=-1)
    return g / (1.0 + torch.exp(-g)) * u


def _gated(s):
    gu = _dequant_rows(s["a"], s["sa"]) @ _dequant_blocks(s["w"], s["sw"]).t()
    h = _activate(gu)
    form = s["case"]["form"]
    if form == "quant":
        return _quant_rows(h)
    return h.to(torch.bfloat16) if form == "bf16" else (h.to(torch.bfloat16), gu.to(torch.bfloat16))


def _experts(s):
    case, off = s["case"], s["offsets"].long()
    r = torch.arange(case["rows"], device="cuda")
    g = torch.searchsorted(off, r, right=True) - 1  # the expert of each row
    at = g * s["most"] + r - off[g]
    a = torch.zeros((case["G"] * s["most"], case["K"]), device="cuda")
    a[at] = _dequant_rows(s["a"], s["sa"])[s["rows"].long()]
    a = a.view(case["G"], s["most"], case["K"]).transpose(1, 2).contiguous()
    gu = torch.bmm(_dequant_blocks(s["w"], s["sw"]), a)  # [G, 2I, most]
    gu = gu.transpose(1, 2).reshape(case["G"] * s["most"], 2 * case["I"])[at]
    return _activate(gu).to(torch.bfloat16)


def _gated_grad(s):
    pow2 = s["case"]["pow2"]
    dh = s["dh"].float()
    g, u = s["gu"].float().chunk(2, dim=1)
    p = 1.0 / (1.0 + torch.exp(-g))
    d = torch.cat([dh * u * p * (1.0 + g * (1.0 - p)), dh * g * p], dim=1)
    out = {"rows": _quant_rows(d, pow2)}
    if s["case"]["M"] % 128 == 0:
        out["columns"] = _quant_rows(d.t().contiguous(), pow2)
        out["h columns"] = _quant_rows((g * p * u).t().contiguous(), pow2)
    return out


def _clip(s):
    norm = torch.stack([g.float().square().sum() for g in s["grads"]]).sum().sqrt()
    c = torch.where(norm <= 1.0, torch.ones_like(norm), 1.0 / norm)
    return {"norm": norm, "grads": [(g.float() * c).to(g.dtype) for g in s["grads"]]}


PLAIN = {"norm": _norm, "norm_grad": _norm_grad, "gated": _gated, "experts": _experts, "gated_grad": _gated_grad,
         "clip": _clip}


# ------------------------------------------------------------------ the library's operators
def _float8(pair):
    return pair[0].view(torch.float8_e4m3fn), pair[1]


def _library(s):
    from fp8_fine_grained_amd import layer

    case = s["case"]
    op = case["op"]
    if op == "norm":
        h, q, scales, rstd = layer.fp8_add_rmsnorm_quant_1x128(s["x"], s["w"], residual=s["r"], eps=EPS,
                                                               pow2=case["pow2"])
        return {"h": h, "q": q.view(torch.float8_e4m3fn), "scales": scales, "rstd": rstd}
    if op == "norm_grad":
        dx, dw = layer.fp8_rmsnorm_backward(s["dy"], s["h"], s["rstd"], s["w"], dh=s["dh"])
        return {"dx": dx, "dw": dw}
    if op == "gated":
        if case["form"] == "quant":
            return _float8(layer.fp8_block_gated_gemm_quant(s["a"], s["sa"], s["w"], s["sw"], accum="exact"))
        return layer.fp8_block_gated_gemm(s["a"], s["sa"], s["w"], s["sw"], save=case["form"] == "saved")
    if op == "experts":
        return layer.fp8_block_grouped_gated_gemm(s["a"], s["sa"], s["offsets"], s["w"], s["sw"],
                                                  row_index=s["rows"])
    if op == "gated_grad":
        columns = case["M"] % 128 == 0
        r = layer.fp8_gated_backward_quant(s["dh"], s["gu"], pow2=case["pow2"], columns=columns, h_columns=columns)
        out = {"rows": _float8(r[0:2])}
        if columns:
            out["columns"], out["h columns"] = _float8(r[2:4]), _float8(r[4:6])
        return out
    return {"norm": layer.clip_grad_norm(s["grads"], 1.0, out=s["out"]), "grads": s["out"]}


def run(state):
    return _library(state) if own else PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------ work
def _bytes_of(case):
    return 2 if case["dtype"] == "bf16" else 4


def work(case):
    op = case["op"]
    if op in ("norm", "norm_grad"):
        M, H, e = case["M"], case["H"], _bytes_of(case)
        extra = 1 if case["residual"] else 0
        if op == "norm":  # x (and the residual) read; codes, scales and rstd (and the sum) written
            return {"bytes": M * H * ((1 + 2 * extra) * e + 1 + 4 / 128) + H * e + 4 * M, "flops": 8 * M * H}
        return {"bytes": M * H * (3 + extra) * e + H * (e + 4) + 4 * M, "flops": 12 * M * H}
    if op == "gated":
        M, n, K = case["M"], case["I"], case["K"]
        out = {"bf16": 2 * n, "saved": 6 * n, "quant": n + n // 128 * 4}[case["form"]]
        scales = 4 * (M * (K // 128) + (2 * n // 128) * (K // 128))
        return {"bytes": M * K + 2 * n * K + scales + M * out, "flops": 4 * M * n * K}
    if op == "experts":
        T, R, n, K = case["T"], case["rows"], case["I"], case["K"]
        live = min(case["G"] - case["empty"], R)
        scales = 4 * (min(T, R) * (K // 128) + live * (2 * n // 128) * (K // 128))
        return {"bytes": min(T, R) * K + live * 2 * n * K + scales + 2 * R * n, "flops": 4 * R * n * K}
    if op == "gated_grad":
        M, n, e = case["M"], case["I"], _bytes_of(case)
        codes = 5 if M % 128 == 0 else 2
        return {"bytes": M * n * (3 * e + codes * (1 + 4 / 128)), "flops": 20 * M * n}
    sizes = _tensors(case)
    return {"bytes": 2 * sum(k * dt.itemsize for k, dt in sizes), "flops": 3 * sum(k for k, _ in sizes)}


# ------------------------------------------------------------------ the definitions in 64 bits
def _e4m3(v):
    """Round to nearest E4M3, ties to even, saturating at 448; float64 in and out."""
    _, e = torch.frexp(v)
    step = torch.exp2((e - 1).clamp(min=-6).double() - 3.0)
    return (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _quantised(v, pow2=False):
    """E4M3 values and scales of v [rows, n] in groups of 128 along n."""
    t = v.unflatten(1, (-1, 128))
    top = t.abs().amax(dim=-1)
    if pow2:
        s = torch.where(top > 0, torch.exp2(torch.ceil(torch.log2(top / E4M3_MAX))), torch.zeros_like(top))
        s = torch.where(E4M3_MAX * s / 2 >= top, s / 2, s)  # log2's rounding at exact powers
        s = torch.where(E4M3_MAX * s < top, s * 2, s)
    else:
        s = top / E4M3_MAX
    safe = torch.where(s > 0, s, torch.ones_like(s))
    return _e4m3(t / safe[..., None]).flatten(1), s


def _values(codes, scales, block_rows):
    """Code values times their scales, one scale per 128 columns and `block_rows` rows."""
    v = codes.view(torch.float8_e4m3fn).double().unflatten(-1, (-1, 128)).unflatten(-3, (-1, block_rows))
    return (v * scales.double()[..., :, None, :, None]).flatten(-4, -3).flatten(-2)


def _silu_product(g, u):
    return g * torch.sigmoid(g) * u


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        z = s["x"].double() + (0 if s["r"] is None else s["r"].double())
        rstd = 1.0 / torch.sqrt((z * z).sum(1) / case["H"] + EPS)
        q, scales = _quantised(s["w"].double() * z * rstd.unsqueeze(1), case["pow2"])
        return {"h": z, "q": q, "scales": scales, "rstd": rstd}
    if op == "norm_grad":
        h, dy, rstd = s["h"].double(), s["dy"].double(), s["rstd"].double().unsqueeze(1)
        t = dy * s["w"].double()
        # d/dh of rstd(h) h: rstd t - h rstd^3 <t, h> / H
        dx = rstd * t - h * rstd ** 3 * ((t * h).sum(1, keepdim=True) / case["H"])
        if s["dh"] is not None:
            dx += s["dh"].double()
        return {"dx": dx, "dw": torch.einsum("mh,mh->h", dy, h * rstd)}
    if op == "gated":
        a = _values(s["a"], s["sa"], 1)
        n = case["I"]
        gate = a @ _values(s["w"][:n], s["sw"][: n // 128], 128).t()
        up = a @ _values(s["w"][n:], s["sw"][n // 128:], 128).t()
        h = _silu_product(gate, up)
        if case["form"] == "quant":
            return _quantised(h)
        return h if case["form"] == "bf16" else (h, torch.cat([gate, up], dim=1))
    if op == "experts":
        off, n = s["offsets"].tolist(), case["I"]
        h = torch.zeros((case["rows"], n), dtype=torch.float64, device="cuda")
        a = _values(s["a"], s["sa"], 1)
        for e in range(case["G"]):
            if off[e + 1] > off[e]:
                t = a[s["rows"][off[e]:off[e + 1]].long()] @ _values(s["w"][e], s["sw"][e], 128).t()
                h[off[e]:off[e + 1]] = _silu_product(t[:, :n], t[:, n:])
        return h
    if op == "gated_grad":
        dh, n = s["dh"].double(), case["I"]
        g, u = s["gu"][:, :n].double(), s["gu"][:, n:].double()
        p = torch.sigmoid(g)
        silu = g * p
        d = torch.cat([dh * u * (p + silu * (1 - p)), dh * silu], dim=1)
        out = {"rows": _quantised(d, case["pow2"])}
        if case["M"] % 128 == 0:
            out["columns"] = _quantised(d.t(), case["pow2"])
            out["h columns"] = _quantised((silu * u).t(), case["pow2"])
        return out
    norm = math.sqrt(sum(float(g.double().square().sum()) for g in s["grads"]))
    c = 1.0 if norm <= 1.0 else 1.0 / norm
    return {"norm": torch.tensor(norm, dtype=torch.float64), "grads": [g.double() * c for g in s["grads"]]}

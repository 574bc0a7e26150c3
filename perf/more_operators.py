"""Cases of the expert layer's operators: what is measured, in plain torch and in the library.

What stands around the grouped products of a mixture-of-experts layer, in training and for few tokens:

* ``route``  scores of the experts (sigmoid or softmax), balance bias, groups, the k best with their weights, and
             the row segments that the grouped products take; its gradient (``route_grad``);
* ``fp4``    products of few rows with 4-bit weights (E2M1 codes, one power-of-two scale per 32): dense, gated, and
             gated over expert segments (``fp4_experts``);
* ``combine`` the weighted sum of the experts' rows per token, and its gradient (``combine_grad``), in the rows'
             type or left 1x128-quantised.

With ``own`` false, ``run`` computes them by elementary torch operations in 32 bits (choices of experts in 64: scores
next to each other must not change places); with ``own`` true it calls the library.  E4M3 codes are returned as
torch.float8_e4m3fn, the values they stand for.
"""

import math

import torch

own = False

E4M3_MAX = 448.0
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one token's choice of 8 among 256 experts in 8 groups while serving: latency
        {"name": "route token", "op": "route", "T": 1, "E": 256, "k": 8, "groups": 8, "kept": 4, "terms": 2,
         "score": "sigmoid", "bias": True, "renormalise": True, "dtype": "f32", "padded": 0, "first": 0, "G": 256},
        # an odd batch with padded tokens at its end, softmax scores of 60 experts, of which this GPU holds 20
        {"name": "route padded softmax", "op": "route", "T": 1037, "E": 60, "k": 4, "groups": 1, "kept": 1,
         "terms": 1, "score": "softmax", "bias": False, "renormalise": False, "dtype": "bf16", "padded": 90,
         "first": 20, "G": 20},
        # the expert layer's tokens in a training step
        {"name": "route step", "op": "route", "T": 8192, "E": 256, "k": 8, "groups": 8, "kept": 4, "terms": 2,
         "score": "sigmoid", "bias": True, "renormalise": True, "dtype": "f32", "padded": 0, "first": 0, "G": 256},
        # the same tokens in the backward pass
        {"name": "route gradient", "op": "route_grad", "T": 8192, "E": 256, "k": 8, "score": "sigmoid",
         "renormalise": True, "dtype": "f32", "balance": False},
        # softmax scores with the gradient of a balance loss on them
        {"name": "route gradient softmax", "op": "route_grad", "T": 333, "E": 60, "k": 4, "score": "softmax",
         "renormalise": False, "dtype": "bf16", "balance": True},
        # a few tokens' experts put together while serving, added to the shared expert's output
        {"name": "combine tokens", "op": "combine", "T": 4, "k": 8, "H": 7168, "dtype": "bf16", "base": True,
         "drop": 0.0},
        # the expert layer's tokens in a training step
        {"name": "combine step", "op": "combine", "T": 8192, "k": 8, "H": 7168, "dtype": "bf16", "base": True,
         "drop": 0.0},
        # its gradient for fp32 rows of a narrow model, where some experts live on other GPUs
        {"name": "combine gradient dropped f32", "op": "combine_grad", "T": 777, "k": 3, "H": 1160, "dtype": "f32",
         "drop": 0.4, "quant": False},
        # its gradient in a training step, quantised for the experts' data gradient
        {"name": "combine gradient quantised", "op": "combine_grad", "T": 8192, "k": 8, "H": 7168, "dtype": "bf16",
         "drop": 0.0, "quant": True},
        # one token through an expert-sized pair of projections while serving
        {"name": "fp4 gated token", "op": "fp4", "M": 1, "N": 4096, "K": 7168, "x": "bf16", "gated": True},
        # a batch of single tokens through a dense down projection, activations quantised already
        {"name": "fp4 batch", "op": "fp4", "M": 48, "N": 7168, "K": 18432, "x": "e4m3", "gated": False},
        # a batch's tokens at one GPU's share of the experts, some of them empty, rows read by index
        {"name": "fp4 experts", "op": "fp4_experts", "T": 128, "rows": 128, "G": 32, "empty": 3, "N": 4096,
         "K": 7168, "x": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _log_of(rng, step, lo, hi):
    """A multiple of `step` in [lo, hi]."""
    return step * _log_int(rng, max(1, lo // step), max(1, hi // step))


def draw(rng):
    op = rng.choice(["route", "route", "route_grad", "combine", "combine_grad", "fp4", "fp4", "fp4_experts"])
    if op in ("route", "route_grad"):
        groups = rng.choice([1, 1, 4, 8]) if op == "route" else 1
        size = _log_int(rng, 4, 512 // groups)
        E = groups * size
        kept = rng.randint(1, groups)
        k = rng.randint(1, min(12, kept * size))
        T = _log_int(rng, 1, 16384)
        case = {"op": op, "T": T, "E": E, "k": k, "score": rng.choice(["sigmoid", "softmax"]),
                "renormalise": rng.random() < 0.6, "dtype": rng.choice(["bf16", "f32"])}
        if op == "route":
            G = rng.choice([E, max(1, E // 4)])
            case.update(groups=groups, kept=kept, terms=rng.randint(1, 2), bias=rng.random() < 0.6,
                        padded=rng.choice([0, T // 9]), first=rng.randint(0, E - G), G=G)
        else:
            case["balance"] = rng.random() < 0.4
        return case
    if op in ("combine", "combine_grad"):
        k = rng.randint(1, 10)
        quant = op == "combine_grad" and rng.random() < 0.5
        H = _log_of(rng, 128 if quant else 8, 128, 8192)
        case = {"op": op, "T": _log_int(rng, 1, max(1, (1 << 28) // (H * k))), "k": k, "H": H,
                "dtype": rng.choice(["bf16", "f32"]), "drop": rng.choice([0.0, 0.5])}
        case.update({"quant": quant} if op == "combine_grad" else {"base": rng.random() < 0.5})
        return case
    K = _log_of(rng, 128, 256, 18432)
    x = rng.choice(["bf16", "e4m3"])
    if op == "fp4":
        gated = rng.random() < 0.5
        N = _log_of(rng, 2 if gated else 1, 64, min(36864, 7168 * 18432 // K))
        return {"op": op, "M": _log_int(rng, 1, 64), "N": N, "K": K, "x": x, "gated": gated}
    G = _log_int(rng, 2, 64)
    N = _log_of(rng, 2, 64, max(64, min(8192, 32 * 4096 * 7168 // (G * K))))
    T = _log_int(rng, 1, 128)
    return {"op": op, "T": T, "rows": T * rng.randint(1, 2), "G": G, "empty": rng.randint(0, G // 2), "N": N, "K": K,
            "x": x}


# ------------------------------------------------------------------ inputs
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(gen, shape, std=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=gen, device="cuda") * std).to(dtype)


def _outliers(gen, x, share=0.001, factor=30.0):
    """Some entries enlarged, as the channels of a residual stream have them."""
    return torch.where(torch.rand(x.shape, generator=gen, device="cuda") < share, x * factor, x)


def _quant_rows(x):
    """1x128 E4M3 codes (float8) and scales of x [M, K] in 32 bits."""
    g = x.float().reshape(x.shape[0], -1, 128)
    s = g.abs().amax(dim=2) / E4M3_MAX
    inv = torch.where(s == 0, torch.zeros_like(s), 1.0 / s)
    return (g * inv[:, :, None]).to(torch.float8_e4m3fn).reshape(x.shape), s


def _fp4_weights(gen, rows, K):
    """E2M1 codes [rows, K/2] and E8M0 scales [rows, K/32] of a weight ~ N(0, 0.02), a few rows at a time."""
    q = torch.empty((rows, K // 2), dtype=torch.uint8, device="cuda")
    s = torch.empty((rows, K // 32), dtype=torch.uint8, device="cuda")
    borders = torch.tensor([(a + b) / 2 for a, b in zip(E2M1, E2M1[1:])], device="cuda")
    step = max(1, (1 << 26) // K)
    for r in range(0, rows, step):
        w = _normal(gen, (min(step, rows - r), K), 0.02).view(-1, K // 32, 32)
        m, e = torch.frexp(w.abs().amax(dim=2))  # amax = m 2^e; 6 = 0.75 * 2^3
        e = (e - 3 + (m > 0.75).to(e.dtype)).clamp(min=-126)
        v = torch.ldexp(w, -e[:, :, None])
        code = torch.bucketize(v.abs(), borders).to(torch.uint8) | ((v < 0).to(torch.uint8) << 3)
        code = code.view(-1, K // 2, 2)
        q[r:r + step] = code[:, :, 0] | (code[:, :, 1] << 4)
        s[r:r + step] = (e + 127).to(torch.uint8)
    return q, s


def _plan(gen, T, k, drop):
    """Rows of T tokens' k experts in (expert, token) order: positions int32 [T, k] (-1: on another GPU), their number."""
    choice = torch.rand((T, max(2 * k, 16)), generator=gen, device="cuda").argsort(dim=1)[:, :k].flatten()
    n = choice.numel()
    gone = torch.randperm(n, generator=gen, device="cuda") < int(drop * n)
    order = (choice + gone * max(n, 2 * k, 16)).argsort(stable=True)  # (dropped ones behind every kept one)
    positions = torch.empty_like(choice)
    positions[order] = torch.arange(n, device="cuda")
    return torch.where(gone, -1, positions).to(torch.int32).view(T, k), n - int(drop * n)


def _routed(gen, case):
    """offsets int32 [G + 1] and row_index int32 [rows] of the experts' case, and the longest segment."""
    live = torch.randperm(case["G"], generator=gen, device="cuda")[: case["G"] - case["empty"]]
    pick = torch.randint(0, len(live), (case["rows"],), generator=gen, device="cuda")
    counts = torch.bincount(live[pick], minlength=case["G"])
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    rows = torch.randint(0, case["T"], (case["rows"],), generator=gen, device="cuda").to(torch.int32)
    return offsets, rows, int(counts.max())


def _mix(gen, T, k):
    """Weights of a token's experts, as a router gives them: they sum to 2.5."""
    w = torch.rand((T, k), generator=gen, device="cuda") + 0.05
    return 2.5 * w / w.sum(dim=1, keepdim=True)


def prepare(case, seed):
    gen = _generator(seed)
    op, s = case["op"], {"case": case}
    if op in ("route", "route_grad"):
        T, E, k = case["T"], case["E"], case["k"]
        s["z"] = _normal(gen, (T, E), 1.0, DTYPES[case["dtype"]])
        if op == "route":
            s["bias"] = (torch.rand(E, generator=gen, device="cuda") - 0.5) * 0.02 if case["bias"] else None
            s["mask"] = torch.arange(T, device="cuda") < T - case["padded"] if case["padded"] else None
        else:
            s["experts"] = torch.rand((T, E), generator=gen, device="cuda").argsort(dim=1)[:, :k].to(torch.int32)
            s["dw"] = _normal(gen, (T, k), 1e-2)
            s["ds"] = _normal(gen, (T, E), 1e-3) if case["balance"] else None
    elif op in ("combine", "combine_grad"):
        T, k, H, dt = case["T"], case["k"], case["H"], DTYPES[case["dtype"]]
        s["positions"], R = _plan(gen, T, k, case["drop"])
        s["w"] = _mix(gen, T, k)
        s["rows"] = _normal(gen, (R, H), 1.0, dt)
        if op == "combine":
            s["base"] = _normal(gen, (T, H), 1.0, dt) if case["base"] else None
        else:
            s["dy"] = _normal(gen, (T, H), 1e-3, dt)
    else:
        rows = case["M"] if op == "fp4" else case["T"]
        x = _outliers(gen, _normal(gen, (rows, case["K"])))
        if case["x"] == "bf16":
            s["x"], s["sx"] = x.to(torch.bfloat16), None
        else:
            q, s["sx"] = _quant_rows(x)
            s["x"] = q.view(torch.uint8)
        G = 1 if op == "fp4" else case["G"]
        w, sw = _fp4_weights(gen, G * case["N"], case["K"])
        if op == "fp4":
            s["w"], s["sw"] = w, sw
        else:
            s["w"], s["sw"] = w.view(G, case["N"], -1), sw.view(G, case["N"], -1)
            s["offsets"], s["rows"], s["most"] = _routed(gen, case)
    return s


# ------------------------------------------------------------------ plain forms (32 bits)
def _scores(z, score):
    if score == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-z))
    e = torch.exp(z - z.amax(dim=1, keepdim=True))
    return e / e.sum(dim=1, keepdim=True)


def _best(c, n):
    """Indices of the n largest of each row, descending, ties to the lowest."""
    return torch.sort(c, dim=1, descending=True, stable=True)[1][:, :n]


def _route(s):
    case, z = s["case"], s["z"]
    T, E, k = case["T"], case["E"], case["k"]
    c = _scores(z.double(), case["score"])  # (64 bits: the choice must not depend on the rounding of a score)
    if s["bias"] is not None:
        c = c + s["bias"].double()
    if case["groups"] > 1:
        g = c.view(T, case["groups"], -1)
        keep = _best(torch.sort(g, dim=2, descending=True)[0][:, :, :case["terms"]].sum(dim=2), case["kept"])
        out = torch.ones((T, case["groups"]), dtype=torch.bool, device=z.device).scatter(1, keep, False)
        c = torch.where(out[:, :, None], -math.inf, g).view(T, E)
    experts = _best(c, k)
    w = torch.gather(_scores(z.float(), case["score"]), 1, experts)
    if case["renormalise"]:
        w = w / w.sum(dim=1, keepdim=True)
    w = w * 2.5
    if s["mask"] is not None:
        experts = torch.where(s["mask"][:, None], experts, -1)
        w = torch.where(s["mask"][:, None], w, 0.0)
    return {"experts": experts.to(torch.int32), "weights": w, **_segments(experts, case["first"], case["G"], k)}


def _segments(experts, first, G, k):
    local = experts.flatten() - first
    key = torch.where((local >= 0) & (local < G), local, G)
    order = key.argsort(stable=True)
    counts = (key[:, None] == torch.arange(G, device=key.device)).sum(dim=0)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    at = torch.arange(key.numel(), device=key.device)
    positions = torch.empty_like(order)
    positions[order] = torch.where(at < offsets[-1], at, -1)
    row_index = torch.where(at < offsets[-1], order // k, 0)
    return {"offsets": offsets.to(torch.int32), "row_index": row_index.to(torch.int32),
            "positions": positions.view(-1, k).to(torch.int32)}


def _route_grad(s):
    case, z, at = s["case"], s["z"].float(), s["experts"].long()
    p = _scores(z, case["score"])
    chosen = torch.gather(p, 1, at)
    dw = s["dw"] * 2.5
    if case["renormalise"]:
        w = chosen / chosen.sum(dim=1, keepdim=True)
        dw = (dw - (dw * w).sum(dim=1, keepdim=True)) / chosen.sum(dim=1, keepdim=True)
    ds = torch.zeros_like(p).scatter(1, at, dw)
    if s["ds"] is not None:
        ds = ds + s["ds"]
    if case["score"] == "sigmoid":
        dz = ds * p * (1.0 - p)
    else:
        dz = p * (ds - (ds * p).sum(dim=1, keepdim=True))
    return dz.to(s["z"].dtype)


def _combine(s):
    y = 0.0 if s["base"] is None else s["base"].float()
    for p, w in zip(s["positions"].t(), s["w"].t()):
        y = y + torch.where(p[:, None] >= 0, s["rows"][p.long().clamp(min=0)].float() * w[:, None], 0.0)
    return y.to(s["rows"].dtype)


def _combine_grad(s):
    case, rows, dy = s["case"], s["rows"], s["dy"].float()
    R, H = rows.shape
    if case["quant"]:
        out = torch.zeros((R + 1, H), dtype=torch.uint8, device=dy.device), torch.zeros((R + 1, H // 128),
                                                                                      device=dy.device)
    else:
        out = (torch.zeros((R + 1, H), dtype=rows.dtype, device=dy.device),)
    dw = []
    for p, w in zip(s["positions"].t(), s["w"].t()):
        at = torch.where(p >= 0, p, R).long()  # (row R takes what belongs nowhere)
        d = dy * w[:, None]
        values = _quant_rows(d) if case["quant"] else (d.to(rows.dtype),)
        out[0][at] = values[0].view(torch.uint8) if case["quant"] else values[0]
        if case["quant"]:
            out[1][at] = values[1]
        dw.append(torch.where(p >= 0, (dy * rows[p.long().clamp(min=0)].float()).sum(dim=1), 0.0))
    dw = torch.stack(dw, dim=1)
    if case["quant"]:
        return {"rows": out[0][:R].view(torch.float8_e4m3fn), "scales": out[1][:R], "weights": dw}
    return {"rows": out[0][:R], "weights": dw}


def _fp4_values(w, sw):
    table = torch.tensor([*E2M1, *[-v for v in E2M1]], device=w.device)
    v = table[torch.stack([w & 15, w >> 4], dim=-1).int()].flatten(-2)
    scale = torch.ldexp(torch.ones((), device=w.device), sw.int() - 127)
    return (v.unflatten(-1, (-1, 32)) * scale[..., None]).flatten(-2)


def _x_values(s):
    if s["sx"] is None:
        return s["x"].float()
    return s["x"].view(torch.float8_e4m3fn).float() * s["sx"].repeat_interleave(128, dim=1)


def _activate(gu):
    g, u = gu.chunk(2, dim=-1)
    return g / (1.0 + torch.exp(-g)) * u


def _fp4(s):
    y = _x_values(s) @ _fp4_values(s["w"], s["sw"]).t()
    return (_activate(y) if s["case"]["gated"] else y).to(torch.bfloat16)


def _fp4_experts(s):
    case, off, most = s["case"], s["offsets"].long(), s["most"]
    r = torch.arange(case["rows"], device="cuda")
    g = torch.searchsorted(off, r, right=True) - 1  # the expert of each row
    at = g * most + r - off[g]
    x = torch.zeros((case["G"] * most, case["K"]), device="cuda")
    x[at] = _x_values(s)[s["rows"].long()]
    x = x.view(case["G"], most, case["K"]).transpose(1, 2).contiguous()
    gu = torch.bmm(_fp4_values(s["w"], s["sw"]), x)  # [G, N, most]
    return _activate(gu.transpose(1, 2).reshape(case["G"] * most, case["N"])[at]).to(torch.bfloat16)


PLAIN = {"route": _route, "route_grad": _route_grad, "combine": _combine, "combine_grad": _combine_grad, "fp4": _fp4,
         "fp4_experts": _fp4_experts}


# ------------------------------------------------------------------ the library's operators
def _library(s):
    from fp8_fine_grained_amd import experts as ex

    case = s["case"]
    op = case["op"]
    if op == "route":
        chosen, weights = ex.route_experts(
            s["z"], case["k"], bias=s["bias"], mask=s["mask"], score=case["score"], groups=case["groups"],
            groups_kept=case["kept"], group_terms=case["terms"], renormalise=case["renormalise"], scale=2.5)
        offsets, row_index, positions = ex.expert_segments(chosen, case["G"], first=case["first"])
        return {"experts": chosen, "weights": weights, "offsets": offsets, "row_index": row_index,
                "positions": positions}
    if op == "route_grad":
        return ex.route_experts_backward(s["dw"], s["experts"], s["z"], score=case["score"],
                                         renormalise=case["renormalise"], scale=2.5, dscores=s["ds"])
    if op == "combine":
        return ex.combine_experts(s["rows"], s["positions"], s["w"], base=s["base"])
    if op == "combine_grad":
        if case["quant"]:
            q, scales, dw = ex.combine_experts_backward_quant(s["dy"], s["positions"], s["w"], rows=s["rows"])
            return {"rows": q.view(torch.float8_e4m3fn), "scales": scales, "weights": dw}
        d, dw = ex.combine_experts_backward(s["dy"], s["positions"], s["w"], rows=s["rows"])
        return {"rows": d, "weights": dw}
    if op == "fp4":
        call = ex.fp4_gated_gemm if case["gated"] else ex.fp4_gemm
        return call(s["x"], s["w"], s["sw"], sx=s["sx"])
    return ex.fp4_grouped_gated_gemm(s["x"], s["offsets"], s["w"], s["sw"], sx=s["sx"], row_index=s["rows"])


def run(state):
    return _library(state) if own else PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------ work
def work(case):
    op = case["op"]
    if op in ("route", "route_grad"):
        T, E, k, e = case["T"], case["E"], case["k"], 2 if case["dtype"] == "bf16" else 4
        if op == "route":  # logits (and bias) read; experts, weights, row_index, positions and offsets written
            return {"bytes": T * E * e + 16 * T * k + 4 * (case["G"] + 1) + (4 * E if case["bias"] else 0),
                    "flops": 8 * T * E}
        return {"bytes": T * E * (2 * e + (4 if case["balance"] else 0)) + 8 * T * k, "flops": 10 * T * E}
    if op in ("combine", "combine_grad"):
        T, k, H, e = case["T"], case["k"], case["H"], 2 if case["dtype"] == "bf16" else 4
        n = T * k - int(case["drop"] * T * k)
        if op == "combine":
            return {"bytes": (n + T * (2 if case["base"] else 1)) * H * e + 8 * T * k, "flops": 2 * n * H}
        out = 1 + 4 / 128 if case["quant"] else e
        return {"bytes": (n * (e + out) + T * e) * H + 12 * T * k, "flops": 4 * n * H}
    N, K = case["N"], case["K"]
    xe = 2 if case["x"] == "bf16" else 1 + 4 / 128
    weight = N * K * (0.5 + 1 / 32)
    if op == "fp4":
        M = case["M"]
        return {"bytes": weight + M * K * xe + M * N * (1 if case["gated"] else 2), "flops": 2 * M * N * K}
    R, live = case["rows"], min(case["G"] - case["empty"], case["rows"])
    return {"bytes": live * weight + min(case["T"], R) * K * xe + R * N, "flops": 2 * R * N * K}


# ------------------------------------------------------------------ the definitions in 64 bits
def _e4m3(v):
    """Round to nearest E4M3, ties to even, saturating at 448; float64 in and out."""
    _, e = torch.frexp(v)
    step = torch.exp2((e - 1).clamp(min=-6).double() - 3.0)
    return (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_scores(z, score):
    return torch.sigmoid(z) if score == "sigmoid" else torch.exp(z - torch.logsumexp(z, dim=1, keepdim=True))


def _exact_route(s, case):
    z = s["z"].double()
    T, E, k = case["T"], case["E"], case["k"]
    p = _exact_scores(z, case["score"])
    c = p if s["bias"] is None else p + s["bias"].double()[None]
    size = E // case["groups"]
    if case["groups"] > 1:
        top = torch.zeros((T, case["groups"]), dtype=torch.float64, device="cuda")
        rest = c.view(T, case["groups"], size).clone()
        for _ in range(case["terms"]):  # the largest, taken out, then the largest again
            best, where = rest.max(dim=2)
            top += best
            rest.scatter_(2, where[:, :, None], -math.inf)
        worse = torch.zeros_like(top, dtype=torch.long)
        for g in range(case["groups"]):  # how many groups come before each
            t = top[:, g:g + 1]
            worse += (t > top) | ((t == top) & (torch.arange(case["groups"], device="cuda") > g))
        c = torch.where((worse < case["kept"]).repeat_interleave(size, dim=1), c, -math.inf)
    left, experts = c.clone(), []
    index = torch.arange(E, device="cuda")
    for _ in range(k):
        e = torch.where(left == left.amax(dim=1, keepdim=True), index, E).amin(dim=1, keepdim=True)
        experts.append(e)
        left.scatter_(1, e, -math.inf)
    experts = torch.cat(experts, dim=1)
    w = p.gather(1, experts)
    w = 2.5 * w / (w.sum(1, keepdim=True) if case["renormalise"] else 1.0)
    live = torch.ones(T, dtype=torch.bool, device="cuda") if s["mask"] is None else s["mask"]
    experts, w = experts.masked_fill(~live[:, None], -1), w.masked_fill(~live[:, None], 0.0)
    # rows in the order of (expert, token, place): how many entries come before each
    flat = experts.flatten() - case["first"]
    here = (flat >= 0) & (flat < case["G"])
    n = T * k
    code = torch.where(here, flat * n, case["G"] * n) + torch.arange(n, device="cuda")
    ranked = torch.sort(code)[0]
    positions = torch.where(here, torch.searchsorted(ranked, code), -1)
    offsets = torch.searchsorted(ranked, torch.arange(case["G"] + 1, device="cuda") * n)
    row_index = torch.zeros(n, dtype=torch.long, device="cuda")
    row_index[positions[here]] = torch.arange(n, device="cuda")[here] // k
    return {"experts": experts.int(), "weights": w, "offsets": offsets.int(), "row_index": row_index.int(),
            "positions": positions.view(T, k).int()}


def _exact_route_grad(s, case):
    """From the Jacobians: dw/ds of the chosen scores, then ds/dz of the row."""
    p = _exact_scores(s["z"].double(), case["score"])
    at = s["experts"].long()
    q, g = p.gather(1, at), 2.5 * s["dw"].double()
    if case["renormalise"]:
        r = q.sum(1, keepdim=True)
        g = g / r - (g * q).sum(1, keepdim=True) / r ** 2
    ds = torch.zeros_like(p)
    ds.scatter_add_(1, at, g)
    if s["ds"] is not None:
        ds += s["ds"].double()
    if case["score"] == "sigmoid":
        return ds * p * torch.sigmoid(-s["z"].double())
    return ds * p - p * torch.einsum("te,te->t", ds, p)[:, None]


def _exact_fp4(w, sw):
    code = torch.stack([w & 15, w >> 4], dim=-1).flatten(-2).long()
    e, m = (code >> 1) & 3, (code & 1).double()
    v = torch.where(e == 0, m / 2, (1 + m / 2) * torch.exp2(e.double() - 1))
    v = torch.where(code >= 8, -v, v)
    return v * torch.exp2(sw.double() - 127).repeat_interleave(32, dim=-1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        return _exact_route(s, case)
    if op == "route_grad":
        return _exact_route_grad(s, case)
    if op == "combine":
        y = torch.zeros((case["T"], case["H"]), dtype=torch.float64, device="cuda")
        for j in range(case["k"]):
            t = (s["positions"][:, j] >= 0).nonzero().flatten()
            y[t] += s["w"][t, j, None].double() * s["rows"][s["positions"][t, j].long()].double()
        return y if s["base"] is None else y + s["base"].double()
    if op == "combine_grad":
        R, dy = s["rows"].shape[0], s["dy"].double()
        rows = torch.zeros((R, case["H"]), dtype=torch.float64, device="cuda")
        dw = torch.zeros((case["T"], case["k"]), dtype=torch.float64, device="cuda")
        for j in range(case["k"]):
            t = (s["positions"][:, j] >= 0).nonzero().flatten()
            at = s["positions"][t, j].long()
            rows[at] = s["w"][t, j, None].double() * dy[t]
            dw[t, j] = torch.einsum("th,th->t", dy[t], s["rows"][at].double())
        if not case["quant"]:
            return {"rows": rows, "weights": dw}
        scales = rows.unflatten(1, (-1, 128)).abs().amax(dim=2) / E4M3_MAX
        safe = torch.where(scales > 0, scales, 1.0)
        return {"rows": _e4m3(rows.div_(safe.repeat_interleave(128, dim=1))), "scales": scales, "weights": dw}
    x = s["x"].double() if s["sx"] is None else (
        s["x"].view(torch.float8_e4m3fn).double() * s["sx"].double().repeat_interleave(128, dim=1))

    def product(rows, w, sw, gated):
        y = rows @ _exact_fp4(w, sw).t()
        if not gated:
            return y
        g, u = y[:, :case["N"] // 2], y[:, case["N"] // 2:]
        return g * torch.sigmoid(g) * u

    if op == "fp4":
        return product(x, s["w"], s["sw"], case["gated"])
    off = s["offsets"].tolist()
    out = torch.zeros((case["rows"], case["N"] // 2), dtype=torch.float64, device="cuda")
    for e in range(case["G"]):
        if off[e + 1] > off[e]:
            out[off[e]:off[e + 1]] = product(x[s["rows"][off[e]:off[e + 1]].long()], s["w"][e], s["sw"][e], True)
    return out

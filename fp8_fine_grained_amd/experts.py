"""ctypes binding of the expert layer's operators of libfp8fg.so (include/fp8fg_experts.h).

What stands around the grouped products of a mixture-of-experts layer: routing and its
gradient, the row segments that the grouped products take, products of few rows with 4-bit
weights, and the combination of the experts' rows with its gradient.  The same names and the
same rules as :mod:`fp8_fine_grained_amd.layer`: torch tensors are device memory, outputs
are allocated when none are given, every step runs in the library's HIP kernels on torch's
current stream (or ``stream=``), there is no fallback, and a refused call raises
:class:`binding.Fp8fgError`.  A call's tensors have to be on one GPU, which need not be the
current one.

    experts, weights = route_experts(logits, 8, bias=bias, groups=8, groups_kept=4)
    offsets, row_index, positions = expert_segments(experts, G)
    h = fp4_grouped_gated_gemm(x, offsets, w13, s13, row_index=row_index)   # or the FP8 products
    rows = fp4_grouped_gemm(h, offsets, w2, s2)
    y = combine_experts(rows, positions, weights, base=shared)
"""

import ctypes
import os

import torch

from . import binding, layer
from .binding import _check, _contig, _dtype_code, _on_stream
from .layer import _elsewhere, _given, _ld, _over_there, _ptr, _rows, _stream, _workspace

HEADER = os.path.join(os.path.dirname(binding.HEADER), "fp8fg_experts.h")

SOFTMAX, SIGMOID = 0, 1

_c = ctypes
_p, _i, _l, _f = _c.c_void_p, _c.c_int, _c.c_int64, _c.c_float
_SIGS = {
    "fp8fg_route_experts": ([_p, _i, _l, _l, _l, _p, _p, _i, _l, _l, _i, _l, _i, _f, _p, _p, _p, _p], _i),
    "fp8fg_route_experts_backward": ([_p, _p, _p, _i, _l, _l, _l, _i, _l, _i, _f, _p, _p, _p], _i),
    "fp8fg_expert_segments": ([_p, _l, _l, _l, _l, _p, _p, _p, _p, _l, _p], _i),
    "fp8fg_expert_segments_workspace": ([_l, _l, _l], _l),
    "fp8fg_combine_experts": ([_p, _i, _l, _l, _l, _p, _p, _l, _l, _p, _l, _p, _p], _i),
    "fp8fg_combine_experts_backward": ([_p, _p, _i, _l, _l, _l, _l, _p, _p, _l, _l, _p, _p, _p], _i),
    "fp8fg_combine_experts_backward_quant": ([_p, _p, _i, _l, _l, _l, _l, _p, _p, _l, _l, _i, _p, _p, _p, _p], _i),
    "fp4_quant_weight_1x32": ([_p, _i, _l, _l, _l, _p, _p, _p], _i),
    "fp4_gemm": ([_p, _p, _p, _p, _p, _i, _l, _l, _l, _p], _i),
    "fp4_gated_gemm": ([_p, _p, _p, _p, _p, _i, _l, _l, _l, _p], _i),
    "fp4_grouped_gemm": ([_p, _p, _l, _p, _p, _l, _p, _p, _p, _i, _l, _l, _l, _p], _i),
    "fp4_grouped_gated_gemm": ([_p, _p, _l, _p, _p, _l, _p, _p, _p, _i, _l, _l, _l, _p], _i),
}

_lib = None


def lib():
    """The loaded library with this module's functions (raises if it is not built)."""
    global _lib
    if _lib is None:
        L = layer.lib()
        for name, (args, res) in _SIGS.items():
            f = getattr(L, name)
            f.argtypes, f.restype = args, res
        _lib = L
    return _lib


_SCORES = {"softmax": SOFTMAX, "sigmoid": SIGMOID, SOFTMAX: SOFTMAX, SIGMOID: SIGMOID}


# ------------------------------------------------------------------ routing
def route_experts(logits, k, bias=None, mask=None, score="sigmoid", groups=1, groups_kept=1, group_terms=2,
                  renormalise=True, scale=1.0, experts=None, weights=None, scores=None, need_scores=False,
                  stream=None):
    """The k experts of each token and their weights, from ``logits`` [T, E] (row-contiguous).

    ``score`` "sigmoid" or "softmax"; ``bias`` fp32 [E] counts for the choice only; with
    ``groups`` > 1 only the ``groups_kept`` groups of the largest sums of their ``group_terms``
    best are chosen from; ``mask`` bool or uint8 [T]: tokens with 0 get no expert.
    Returns ``(experts int32 [T, k], weights fp32 [T, k])``, and the scores fp32 [T, E] as a
    third with ``need_scores=True`` or a ``scores`` buffer.  Places without an expert hold -1."""
    if stream is not None:
        return _on_stream(stream, route_experts, locals())
    if _elsewhere(logits, bias, mask, experts, weights, scores):
        return _over_there(logits, route_experts, locals())
    _rows(logits)
    T, E = logits.shape
    if bias is not None:
        _given("bias", torch.float32, (E,), bias)
    if mask is not None:
        if mask.dtype not in (torch.bool, torch.uint8) or mask.shape != (T,) or not mask.is_contiguous():
            raise ValueError("mask must be contiguous bool or uint8 [T]")
    if experts is None:
        experts = logits.new_empty((T, k), dtype=torch.int32)
    else:
        _given("experts", torch.int32, (T, k), experts)
    if weights is None:
        weights = logits.new_empty((T, k), dtype=torch.float32)
    else:
        _given("weights", torch.float32, (T, k), weights)
    if scores is not None:
        _given("scores", torch.float32, (T, E), scores)
    elif need_scores:
        scores = logits.new_empty((T, E), dtype=torch.float32)
    st = (_lib or lib()).fp8fg_route_experts(
        logits.data_ptr(), _dtype_code(logits.dtype), T, E, _ld(logits), _ptr(bias), _ptr(mask), _SCORES[score],
        groups, groups_kept, group_terms, k, 1 if renormalise else 0, scale, experts.data_ptr(), weights.data_ptr(),
        _ptr(scores), _stream(logits))
    _check("fp8fg_route_experts", st)
    return (experts, weights) if scores is None else (experts, weights, scores)


def route_experts_backward(dweights, experts, logits, score="sigmoid", renormalise=True, scale=1.0, dscores=None,
                           dlogits=None, stream=None):
    """Gradient of the routing weights with respect to the logits: dlogits [T, E] of logits' type.

    ``dweights`` fp32 [T, k], ``experts`` as :func:`route_experts` returned them; ``dscores``
    fp32 [T, E] is the gradient that arrives at the scores (of a balance loss)."""
    if stream is not None:
        return _on_stream(stream, route_experts_backward, locals())
    if _elsewhere(dweights, experts, logits, dscores, dlogits):
        return _over_there(logits, route_experts_backward, locals())
    _rows(logits, dweights)
    T, E = logits.shape
    k = dweights.shape[1]
    _given("dweights", torch.float32, (T, k), dweights)
    _given("experts", torch.int32, (T, k), experts)
    if dscores is not None:
        _given("dscores", torch.float32, (T, E), dscores)
    if dlogits is None:
        dlogits = logits.new_empty((T, E))
    else:
        _given("dlogits", logits.dtype, (T, E), dlogits)
    st = (_lib or lib()).fp8fg_route_experts_backward(
        dweights.data_ptr(), experts.data_ptr(), logits.data_ptr(), _dtype_code(logits.dtype), T, E, _ld(logits),
        _SCORES[score], k, 1 if renormalise else 0, scale, _ptr(dscores), dlogits.data_ptr(), _stream(logits))
    _check("fp8fg_route_experts_backward", st)
    return dlogits


def expert_segments(experts, G, first=0, offsets=None, row_index=None, positions=None, workspace=None, stream=None):
    """Row segments of the experts first .. first + G - 1 for the grouped products.

    ``experts`` int32 [T, k].  Returns ``(offsets int32 [G+1], row_index int32 [T*k], positions
    int32 [T, k])``: rows in the order of (expert, token, place); row_index holds each row's
    token (0 behind the last segment), positions each entry's row (-1: no local expert)."""
    if stream is not None:
        return _on_stream(stream, expert_segments, locals())
    if _elsewhere(experts, offsets, row_index, positions, workspace):
        return _over_there(experts, expert_segments, locals())
    _rows(experts)
    T, k = experts.shape
    _given("experts", torch.int32, (T, k), experts)
    if offsets is None:
        offsets = experts.new_empty(G + 1)
    else:
        _given("offsets", torch.int32, (G + 1,), offsets)
    if row_index is None:
        row_index = experts.new_empty(T * k)
    else:
        _given("row_index", torch.int32, (T * k,), row_index)
    if positions is None:
        positions = torch.empty_like(experts)
    else:
        _given("positions", torch.int32, (T, k), positions)
    L = _lib or lib()
    ws, nbytes = _workspace(L.fp8fg_expert_segments_workspace(T, k, G), workspace, experts.device)
    st = L.fp8fg_expert_segments(experts.data_ptr(), T, k, first, G, offsets.data_ptr(), row_index.data_ptr(),
                                 positions.data_ptr(), _ptr(ws), nbytes, _stream(experts))
    _check("fp8fg_expert_segments", st)
    return offsets, row_index, positions


# ------------------------------------------------------------------ combination
def _entries(positions, weights):
    """(T, k) of a plan, checked."""
    if positions.dim() != 2:
        raise ValueError("positions must be [T, k]")
    T, k = positions.shape
    _given("positions", torch.int32, (T, k), positions)
    if weights is not None:
        _given("weights", torch.float32, (T, k), weights)
    return T, k


def combine_experts(rows, positions, weights=None, base=None, y=None, stream=None):
    """y[t] = base[t] + sum_j weights[t, j] rows[positions[t, j]], [T, H] of rows' type.

    ``positions`` as :func:`expert_segments` returned them (a value that names no row adds
    nothing); ``weights`` fp32 [T, k], or None for ones: the gradient of the dispatch, with
    the rows' gradients as ``rows``."""
    if stream is not None:
        return _on_stream(stream, combine_experts, locals())
    if _elsewhere(rows, positions, weights, base, y):
        return _over_there(rows, combine_experts, locals())
    _rows(rows, base)
    R, H = rows.shape
    T, k = _entries(positions, weights)
    if base is not None and (base.dtype != rows.dtype or base.shape != (T, H)):
        raise ValueError(f"base must be {rows.dtype} {[T, H]}")
    if y is None:
        y = rows.new_empty((T, H))
    else:
        _given("y", rows.dtype, (T, H), y)
    st = (_lib or lib()).fp8fg_combine_experts(
        rows.data_ptr(), _dtype_code(rows.dtype), R, H, _ld(rows), positions.data_ptr(), _ptr(weights), T, k,
        _ptr(base), _ld(base), y.data_ptr(), _stream(rows))
    _check("fp8fg_combine_experts", st)
    return y


def _combine_backward_sizes(dy, positions, weights, rows, R, dweights, need_dweights):
    """(R, T, k, H, dweights or None) of the combination's gradient."""
    _rows(dy, rows)
    T, k = _entries(positions, weights)
    if dy.shape[0] != T:
        raise ValueError("dy and positions must have one row per token")
    H = dy.shape[1]
    if rows is not None:
        if rows.dtype != dy.dtype or rows.shape[1] != H or (R is not None and rows.shape[0] != R):
            raise ValueError(f"rows must be {dy.dtype} [R, {H}]")
        R = rows.shape[0]
    elif R is None:
        R = T * k
    if dweights is not None:
        _given("dweights", torch.float32, (T, k), dweights)
    elif need_dweights and rows is not None:
        dweights = dy.new_empty((T, k), dtype=torch.float32)
    if dweights is not None and rows is None:
        raise ValueError("dweights needs the rows")
    return R, T, k, H, dweights


def combine_experts_backward(dy, positions, weights=None, rows=None, R=None, drows=None, dweights=None,
                             need_drows=True, need_dweights=True, stream=None):
    """Gradient of :func:`combine_experts`: ``(drows [R, H] of dy's type, dweights fp32 [T, k])``.

    ``rows`` as the forward call took them, for dweights (None without them); R defaults to
    their number, or T * k.  Rows that no position names stay as they were; each row may be
    named once."""
    if stream is not None:
        return _on_stream(stream, combine_experts_backward, locals())
    if _elsewhere(dy, positions, weights, rows, drows, dweights):
        return _over_there(dy, combine_experts_backward, locals())
    if R is None and rows is None and drows is not None:
        R = drows.shape[0]
    R, T, k, H, dweights = _combine_backward_sizes(dy, positions, weights, rows, R, dweights, need_dweights)
    if drows is not None:
        _given("drows", dy.dtype, (R, H), drows)
    elif need_drows:
        drows = dy.new_empty((R, H))
    st = (_lib or lib()).fp8fg_combine_experts_backward(
        dy.data_ptr(), _ptr(rows), _dtype_code(dy.dtype), R, H, _ld(dy), _ld(rows), positions.data_ptr(),
        _ptr(weights), T, k, _ptr(drows), _ptr(dweights), _stream(dy))
    _check("fp8fg_combine_experts_backward", st)
    return drows, dweights


def combine_experts_backward_quant(dy, positions, weights=None, rows=None, R=None, pow2=False, q=None, scales=None,
                                   dweights=None, need_dweights=True, stream=None):
    """The same with the rows' gradient leaving 1x128-quantised: ``(q uint8 [R, H], scales fp32
    [R, H/128], dweights)``, for the data gradient of the experts' products."""
    if stream is not None:
        return _on_stream(stream, combine_experts_backward_quant, locals())
    if _elsewhere(dy, positions, weights, rows, q, scales, dweights):
        return _over_there(dy, combine_experts_backward_quant, locals())
    if R is None and rows is None and q is not None:
        R = q.shape[0]
    R, T, k, H, dweights = _combine_backward_sizes(dy, positions, weights, rows, R, dweights, need_dweights)
    if q is None:
        q = dy.new_empty((R, H), dtype=torch.uint8)
    else:
        _given("q", torch.uint8, (R, H), q)
    if scales is None:
        scales = dy.new_empty((R, H // 128), dtype=torch.float32)
    else:
        _given("scales", torch.float32, (R, H // 128), scales)
    st = (_lib or lib()).fp8fg_combine_experts_backward_quant(
        dy.data_ptr(), _ptr(rows), _dtype_code(dy.dtype), R, H, _ld(dy), _ld(rows), positions.data_ptr(),
        _ptr(weights), T, k, 1 if pow2 else 0, q.data_ptr(), scales.data_ptr(), _ptr(dweights), _stream(dy))
    _check("fp8fg_combine_experts_backward_quant", st)
    return q, scales, dweights


# ------------------------------------------------------------------ 4-bit weights
def fp4_quant_weight_1x32(w, q=None, scales=None, stream=None):
    """4-bit quantisation of ``w`` [N, K], or [G, N, K] over experts, in groups of 32 along K.

    Returns ``(q uint8 [.., N, K/2], scales uint8 [.., N, K/32])``: E2M1 codes, two to a byte
    (the even element low), and E8M0 scale bytes.  A 2-D ``w`` may have any row pitch of whole
    16 bytes; over experts it is contiguous."""
    if stream is not None:
        return _on_stream(stream, fp4_quant_weight_1x32, locals())
    if _elsewhere(w, q, scales):
        return _over_there(w, fp4_quant_weight_1x32, locals())
    if w.dim() == 3:
        _contig(w)
        ld = w.shape[2]
    else:
        _rows(w)
        ld = _ld(w)
    *lead, K = w.shape
    N = lead[0] if len(lead) == 1 else lead[0] * lead[1]
    if K % 128 != 0:  # (the library's own refusal, before a shape could hide it)
        raise binding.Fp8fgError("fp4_quant_weight_1x32", binding.ERR_UNSUPPORTED)
    if q is None:
        q = w.new_empty((*lead, K // 2), dtype=torch.uint8)
    else:
        _given("q", torch.uint8, (*lead, K // 2), q)
    if scales is None:
        scales = w.new_empty((*lead, K // 32), dtype=torch.uint8)
    else:
        _given("scales", torch.uint8, (*lead, K // 32), scales)
    st = (_lib or lib()).fp4_quant_weight_1x32(w.data_ptr(), _dtype_code(w.dtype), N, K, ld, q.data_ptr(),
                                               scales.data_ptr(), _stream(w))
    _check("fp4_quant_weight_1x32", st)
    return q, scales


def _fp4_operands(x, sx, w, sw, experts, gated):
    """(K, N): N columns of the output, after checking the operands against each other."""
    if x.dim() != 2 or w.dim() != (3 if experts else 2):
        raise ValueError("x must be [rows, K], w [N, K/2], or [G, N, K/2] over experts")
    rows, K = x.shape
    if sx is None:
        _given("x", torch.bfloat16, (rows, K), x)
    else:
        _given("x", torch.uint8, (rows, K), x)
        _given("sx", torch.float32, (rows, K // 128), sx)
    lead = w.shape[:-1]
    if K % 128 != 0 or (gated and lead[-1] % 2 != 0):  # (the library's own refusal, before a shape could hide it)
        raise binding.Fp8fgError("4-bit product", binding.ERR_UNSUPPORTED)
    _given("w", torch.uint8, (*lead, K // 2), w)
    _given("sw", torch.uint8, (*lead, K // 32), sw)
    return K, lead[-1] // 2 if gated else lead[-1]


def _fp4_output(rows, N, x, y, out_dtype):
    if y is None:
        return x.new_empty((rows, N), dtype=out_dtype)
    _given("the output", y.dtype, (rows, N), y)
    return y


def _fp4_dense(name, x, sx, w, sw, y, out_dtype, gated):
    K, N = _fp4_operands(x, sx, w, sw, False, gated)
    M = x.shape[0]
    y = _fp4_output(M, N, x, y, out_dtype)
    st = getattr(_lib or lib(), name)(x.data_ptr(), _ptr(sx), w.data_ptr(), sw.data_ptr(), y.data_ptr(),
                                      _dtype_code(y.dtype), M, N, K, _stream(x))
    _check(name, st)
    return y


def _fp4_grouped(name, x, sx, offsets, row_index, w, sw, y, out_dtype, gated):
    K, N = _fp4_operands(x, sx, w, sw, True, gated)
    T, G = x.shape[0], w.shape[0]
    _given("offsets", torch.int32, (G + 1,), offsets)
    M = T
    if row_index is not None:
        if row_index.dim() != 1:
            raise ValueError("row_index must be int32 [M_total]")
        M = row_index.numel()
        _given("row_index", torch.int32, (M,), row_index)
    y = _fp4_output(M, N, x, y, out_dtype)
    st = getattr(_lib or lib(), name)(x.data_ptr(), _ptr(sx), T, _ptr(row_index), offsets.data_ptr(), G, w.data_ptr(),
                                      sw.data_ptr(), y.data_ptr(), _dtype_code(y.dtype), M, N, K, _stream(x))
    _check(name, st)
    return y


def fp4_gemm(x, w, sw, sx=None, out_dtype=torch.bfloat16, y=None, stream=None):
    """Y = X deq(W)^T [M, N] for few rows: ``x`` bf16 [M, K], or E4M3 codes (uint8) with their
    1x128 scales ``sx``; ``w``, ``sw`` as :func:`fp4_quant_weight_1x32` returned them."""
    if stream is not None:
        return _on_stream(stream, fp4_gemm, locals())
    if _elsewhere(x, w, sw, sx, y):
        return _over_there(x, fp4_gemm, locals())
    return _fp4_dense("fp4_gemm", x, sx, w, sw, y, out_dtype, False)


def fp4_gated_gemm(x, w, sw, sx=None, out_dtype=torch.bfloat16, h=None, stream=None):
    """h = g sigmoid(g) u [M, I]; ``w`` [2I, K/2] holds the gate rows, then the up rows."""
    if stream is not None:
        return _on_stream(stream, fp4_gated_gemm, locals())
    if _elsewhere(x, w, sw, sx, h):
        return _over_there(x, fp4_gated_gemm, locals())
    return _fp4_dense("fp4_gated_gemm", x, sx, w, sw, h, out_dtype, True)


def fp4_grouped_gemm(x, offsets, w, sw, sx=None, row_index=None, out_dtype=torch.bfloat16, y=None, stream=None):
    """The product over expert row segments ``offsets`` (device int32 [G+1]) with weights ``w``
    [G, N, K/2]: row r is ``x[row_index[r]]``, or ``x[r]``.  Y [M_total, N] in routed-row order;
    rows behind the last segment stay as they were."""
    if stream is not None:
        return _on_stream(stream, fp4_grouped_gemm, locals())
    if _elsewhere(x, offsets, w, sw, sx, row_index, y):
        return _over_there(x, fp4_grouped_gemm, locals())
    return _fp4_grouped("fp4_grouped_gemm", x, sx, offsets, row_index, w, sw, y, out_dtype, False)


def fp4_grouped_gated_gemm(x, offsets, w, sw, sx=None, row_index=None, out_dtype=torch.bfloat16, h=None, stream=None):
    """The gated pair over expert row segments, ``w`` [G, 2I, K/2]: h [M_total, I]."""
    if stream is not None:
        return _on_stream(stream, fp4_grouped_gated_gemm, locals())
    if _elsewhere(x, offsets, w, sw, sx, row_index, h):
        return _over_there(x, fp4_grouped_gated_gemm, locals())
    return _fp4_grouped("fp4_grouped_gated_gemm", x, sx, offsets, row_index, w, sw, h, out_dtype, True)

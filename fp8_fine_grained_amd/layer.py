"""ctypes binding of the layer operators of libfp8fg.so (include/fp8fg_layer.h).

The operators between the FP8 GEMMs of a feed-forward sublayer, with the same
names and the same rules as :mod:`fp8_fine_grained_amd.binding`: torch tensors
are device memory, outputs are allocated when none are given, every step runs
in the library's HIP kernels on torch's current stream (or ``stream=``), there
is no fallback, and a refused call raises :class:`binding.Fp8fgError`.  A call's
tensors have to be on one GPU, which need not be the current one.

``stream=`` is the same as making the call with that stream current: outputs and
scratch memory that the call allocates come from that stream's memory, and the
outputs may be used on the stream that is current outside.  As in torch, ordering the
two streams, and keeping the inputs until the call's work is done, is the caller's part.
"""

import ctypes
import os
from array import array

import torch

from . import binding
from .binding import _accum_code, _check, _contig, _dtype_code, _on_stream

HEADER = os.path.join(os.path.dirname(binding.HEADER), "fp8fg_layer.h")

_c = ctypes
_p, _i, _l, _f = _c.c_void_p, _c.c_int, _c.c_int64, _c.c_float
_SIGS = {
    "fp8_add_rmsnorm_quant_1x128": ([_p, _p, _i, _l, _l, _l, _l, _p, _i, _f, _i, _p, _p, _p, _p, _p, _p], _i),
    "fp8_rmsnorm_backward": ([_p, _p, _p, _i, _l, _l, _l, _l, _l, _p, _p, _i, _p, _p, _p, _l, _p], _i),
    "fp8_rmsnorm_backward_workspace": ([_l, _l], _l),
    "fp8_block_gated_gemm": ([_p, _p, _p, _p, _i, _p, _i, _p, _l, _l, _l, _p], _i),
    "fp8_block_gated_gemm_quant": ([_p, _p, _p, _p, _i, _i, _p, _p, _p, _p, _l, _l, _l, _l, _p], _i),
    "fp8_block_gated_gemm_quant_workspace": ([_i, _l, _l, _l, _l], _l),
    "fp8_block_grouped_gated_gemm": ([_p, _p, _l, _p, _p, _l, _p, _p, _i, _p, _i, _p, _l, _l, _l, _p], _i),
    "fp8_block_grouped_gated_gemm_quant": ([_p, _p, _l, _p, _p, _l, _p, _p, _i, _i, _p, _p, _p, _p, _l, _l, _l, _l,
                                            _p], _i),
    "fp8_gated_backward_quant": ([_p, _p, _i, _l, _l, _l, _i, _p, _p, _p, _p, _p, _p, _p], _i),
    "fp8fg_grad_norm": ([_p, _p, _p, _l, _p, _p, _l, _p], _i),
    "fp8fg_clip_grad_norm": ([_p, _p, _p, _p, _l, _f, _p, _p, _l, _p], _i),
    "fp8fg_grad_norm_workspace": ([_l], _l),
}

_lib = None


def lib():
    """The loaded library with this module's functions (raises if it is not built)."""
    global _lib
    if _lib is None:
        L = binding.lib()
        for name, (args, res) in _SIGS.items():
            f = getattr(L, name)
            f.argtypes, f.restype = args, res
        _lib = L
    return _lib


# A single token's kernels take a few microseconds, so the calls keep their host side
# short: pointers and the stream go as plain integers, only what a caller passed
# in is checked, and each output is one allocation.
_raw_stream = torch._C._cuda_getCurrentRawStream  # current_stream() without building the object
_current_gpu = torch._C._cuda_getDevice


def _stream(t):
    """torch's current HIP stream on the device of ``t``."""
    return _raw_stream(t.get_device())


def _elsewhere(first, *rest):
    """Whether the tensors (or None), which have to be on one GPU, are on another than the current one."""
    at = first.get_device()
    for t in rest:
        if t is not None and t.get_device() != at:
            raise ValueError("all tensors must be on one GPU")
    if at < 0:
        raise ValueError("all tensors must be on one GPU")
    return at != _current_gpu()


def _over_there(t, call, args):
    """``call(**args)`` with the GPU of ``t`` as the current one, whose kernels are launched."""
    with torch.cuda.device(t.get_device()):
        return call(**args)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _workspace(nbytes, given, device):
    """``given``, or ``nbytes`` of fresh scratch memory of the current stream (which may
    have it back when the call returns: its next user comes after the call's kernels)."""
    if given is not None:
        _contig(given)
        return given, given.numel() * given.element_size()
    if nbytes == 0:
        return None, 0
    return torch.empty(nbytes, dtype=torch.uint8, device=device), nbytes


def _rows(*ts):
    for t in ts:
        if t is not None and (t.dim() != 2 or t.stride(1) != 1):
            raise ValueError("row operands must be 2-D and row-contiguous")


def _ld(t):
    """Row pitch; a single row may carry any stride, so its own length serves."""
    if t is None:
        return 0
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _like(what, dtype, shape, *ts):
    for t in ts:
        if t is not None and (t.dtype != dtype or t.shape != shape):
            raise ValueError(f"{what} must be {dtype} {list(shape)}")


def _given(what, dtype, shape, *ts):
    """Checks of tensors that a kernel takes contiguous: a caller's outputs, saved values."""
    for t in ts:
        if t is not None:
            if t.dtype != dtype or t.shape != shape:
                raise ValueError(f"{what} must be {dtype} {list(shape)}")
            if not t.is_contiguous():
                raise ValueError(f"{what} must be contiguous")


def _weight(w, H):
    if w.shape != (H,) or not w.is_contiguous():
        raise ValueError("weight must be contiguous [H]")


def fp8_add_rmsnorm_quant_1x128(x, weight, residual=None, eps=1e-6, pow2=False, h=None, y=None, q=None, scales=None,
                                rstd=None, stream=None):
    """Residual addition, RMS norm and 1x128 quantisation of ``x`` [M, H] in one pass.

    ``x`` and ``residual`` are row-contiguous (any row pitch of whole 16 bytes).
    Pass ``y`` (of x's type) to also have the normed rows in high precision.
    Returns ``(h, q uint8 [M, H], scales fp32 [M, H/128], rstd fp32 [M])``;
    ``h`` is x + residual rounded to x's type, and x itself without a residual."""
    if stream is not None:
        return _on_stream(stream, fp8_add_rmsnorm_quant_1x128, locals())
    if _elsewhere(x, weight, residual, h, y, q, scales, rstd):
        return _over_there(x, fp8_add_rmsnorm_quant_1x128, locals())
    _rows(x, residual)
    M, H = x.shape
    dt = x.dtype
    _like("residual", dt, (M, H), residual)
    _weight(weight, H)
    if h is not None or y is not None:
        _given("h and y", dt, (M, H), h, y)
    if residual is not None and h is None:
        h = x.new_empty((M, H))
    if q is None:
        q = x.new_empty((M, H), dtype=torch.uint8)
    else:
        _given("q", torch.uint8, (M, H), q)
    if scales is None:
        scales = x.new_empty((M, H // 128), dtype=torch.float32)
    else:
        _given("scales", torch.float32, (M, H // 128), scales)
    if rstd is None:
        rstd = x.new_empty(M, dtype=torch.float32)
    else:
        _given("rstd", torch.float32, (M,), rstd)
    st = (_lib or lib()).fp8_add_rmsnorm_quant_1x128(
        x.data_ptr(), _ptr(residual), _dtype_code(dt), M, H, _ld(x), _ld(residual), weight.data_ptr(),
        _dtype_code(weight.dtype), eps, 1 if pow2 else 0, _ptr(h), _ptr(y), q.data_ptr(), scales.data_ptr(),
        rstd.data_ptr(), _stream(x))
    _check("fp8_add_rmsnorm_quant_1x128", st)
    return x if h is None else h, q, scales, rstd


def fp8_rmsnorm_backward(dy, h, rstd, weight, dh=None, dx=None, dw=None, need_dw=True, workspace=None, stream=None):
    """Gradient of the norm: ``(dx [M, H] of dy's type, dw fp32 [H])``.

    ``h`` and ``rstd`` as the forward call returned them; ``dh`` is the gradient
    that arrives along the residual stream.  ``need_dw=False``: dw is None."""
    if stream is not None:
        return _on_stream(stream, fp8_rmsnorm_backward, locals())
    if _elsewhere(dy, h, rstd, weight, dh, dx, dw, workspace):
        return _over_there(dy, fp8_rmsnorm_backward, locals())
    _rows(dy, h, dh)
    M, H = dy.shape
    _like("h and dh", dy.dtype, (M, H), h, dh)
    _given("rstd", torch.float32, (M,), rstd)
    _weight(weight, H)
    if dx is None:
        dx = dy.new_empty((M, H))
    else:
        _given("dx", dy.dtype, (M, H), dx)
    if dw is not None:
        _given("dw", torch.float32, (H,), dw)
    elif need_dw:
        dw = dy.new_empty(H, dtype=torch.float32)
    L = _lib or lib()
    ws, nbytes = None, 0
    if dw is not None:
        ws, nbytes = _workspace(L.fp8_rmsnorm_backward_workspace(M, H), workspace, dy.device)
    st = L.fp8_rmsnorm_backward(
        dy.data_ptr(), h.data_ptr(), _ptr(dh), _dtype_code(dy.dtype), M, H, _ld(dy), _ld(h), _ld(dh), rstd.data_ptr(),
        weight.data_ptr(), _dtype_code(weight.dtype), dx.data_ptr(), _ptr(dw), _ptr(ws), nbytes, _stream(dy))
    _check("fp8_rmsnorm_backward", st)
    return dx, dw


def _gated_operands(a, sa, w, sw, experts=False):
    """Shapes of a gated product: (K, I) after checking operands against each other."""
    if a.dim() != 2 or w.dim() != (3 if experts else 2):
        raise ValueError("a must be [rows, K], w [2I, K], or [G, 2I, K] over experts")
    rows, K = a.shape
    lead, I2 = w.shape[:-2], w.shape[-2]
    _given("a", torch.uint8, (rows, K), a)
    _given("sa", torch.float32, (rows, K // 128), sa)
    _given("w", torch.uint8, (*lead, I2, K), w)
    if I2 % 256 != 0 or K % 128 != 0:  # (the library's own refusal, before a shape check could hide it)
        raise binding.Fp8fgError("gated product", binding.ERR_UNSUPPORTED)
    _given("sw", torch.float32, (*lead, I2 // 128, K // 128), sw)
    return K, I2 // 2


def _gated_outputs(rows, inner, dtype, a, h, gu, save):
    """h (or its codes, dtype uint8) and gu, allocated beside ``a`` where they are not given."""
    if h is None:
        h = a.new_empty((rows, inner), dtype=dtype)
    else:
        _given("h", h.dtype if dtype != torch.uint8 else dtype, (rows, inner), h)
    if gu is not None or save:
        gu_dtype = torch.bfloat16 if dtype == torch.uint8 else h.dtype
        if gu is None:
            gu = a.new_empty((rows, 2 * inner), dtype=gu_dtype)
        else:
            _given("gu", gu_dtype, (rows, 2 * inner), gu)
    return h, gu


def _scales_out(rows, inner, a, scales):
    if scales is None:
        return a.new_empty((rows, inner // 128), dtype=torch.float32)
    _given("scales", torch.float32, (rows, inner // 128), scales)
    return scales


def fp8_block_gated_gemm(a, sa, w, sw, accum=None, out_dtype=torch.bfloat16, h=None, gu=None, save=False,
                         stream=None):
    """h = g sigmoid(g) u [M, I] with g, u = deq(a) deq(w)^T, in one kernel.

    ``w`` [2I, K] holds the gate rows, then the up rows; ``accum`` as in
    :func:`binding.fp8_block_gemm`.  With ``save=True`` (or a ``gu`` buffer) also
    g and u [M, 2I] for the backward pass: returns ``(h, gu)``, else ``h``."""
    if stream is not None:
        return _on_stream(stream, fp8_block_gated_gemm, locals())
    if _elsewhere(a, sa, w, sw, h, gu):
        return _over_there(a, fp8_block_gated_gemm, locals())
    M = a.shape[0]
    K, inner = _gated_operands(a, sa, w, sw)
    h, gu = _gated_outputs(M, inner, out_dtype, a, h, gu, save)
    st = (_lib or lib()).fp8_block_gated_gemm(
        _ptr(a), _ptr(sa), _ptr(w), _ptr(sw), _accum_code(accum, h.dtype), _ptr(h), _dtype_code(h.dtype), _ptr(gu),
        M, inner, K, _stream(a))
    _check("fp8_block_gated_gemm", st)
    return h if gu is None else (h, gu)


def fp8_block_gated_gemm_quant(a, sa, w, sw, accum="fp8", pow2=False, q=None, scales=None, gu=None, save=False,
                               workspace=None, stream=None):
    """The same with h leaving 1x128-quantised: ``(q uint8 [M, I], scales fp32 [M, I/128])``,
    and the bf16 ``gu`` [M, 2I] as a third with ``save=True``."""
    if stream is not None:
        return _on_stream(stream, fp8_block_gated_gemm_quant, locals())
    if _elsewhere(a, sa, w, sw, q, scales, gu, workspace):
        return _over_there(a, fp8_block_gated_gemm_quant, locals())
    M = a.shape[0]
    K, inner = _gated_operands(a, sa, w, sw)
    q, gu = _gated_outputs(M, inner, torch.uint8, a, q, gu, save)
    scales = _scales_out(M, inner, a, scales)
    mode = _accum_code(accum, torch.bfloat16)
    L = _lib or lib()
    ws, nbytes = _workspace(L.fp8_block_gated_gemm_quant_workspace(mode, M, inner, K, 0), workspace, a.device)
    st = L.fp8_block_gated_gemm_quant(
        _ptr(a), _ptr(sa), _ptr(w), _ptr(sw), mode, 1 if pow2 else 0, _ptr(q), _ptr(scales), _ptr(gu), _ptr(ws),
        nbytes, M, inner, K, _stream(a))
    _check("fp8_block_gated_gemm_quant", st)
    return (q, scales) if gu is None else (q, scales, gu)


def _segments(a, offsets, w, row_index):
    if w.dim() != 3 or offsets.dtype != torch.int32 or offsets.numel() != w.shape[0] + 1:
        raise ValueError("w must be [G, 2I, K] and offsets int32 [G+1]")
    _contig(offsets)
    if row_index is None:
        return a.shape[0]
    if row_index.dtype != torch.int32 or row_index.dim() != 1:
        raise ValueError("row_index must be int32 [M_total]")
    _contig(row_index)
    return row_index.numel()


def fp8_block_grouped_gated_gemm(a, sa, offsets, w, sw, row_index=None, accum=None, out_dtype=torch.bfloat16, h=None,
                                 gu=None, save=False, stream=None):
    """The gated product over expert row segments ``offsets`` (device int32 [G+1]) with
    weights ``w`` [G, 2I, K].  Row r is token ``row_index[r]`` of ``a`` [T, K], or row r
    of ``a`` itself.  Returns ``h`` [M_total, I] (and ``gu``) in routed-row order."""
    if stream is not None:
        return _on_stream(stream, fp8_block_grouped_gated_gemm, locals())
    if _elsewhere(a, sa, offsets, w, sw, row_index, h, gu):
        return _over_there(a, fp8_block_grouped_gated_gemm, locals())
    M = _segments(a, offsets, w, row_index)
    K, inner = _gated_operands(a, sa, w, sw, experts=True)
    h, gu = _gated_outputs(M, inner, out_dtype, a, h, gu, save)
    st = (_lib or lib()).fp8_block_grouped_gated_gemm(
        _ptr(a), _ptr(sa), a.shape[0], _ptr(row_index), _ptr(offsets), w.shape[0], _ptr(w), _ptr(sw),
        _accum_code(accum, h.dtype), _ptr(h), _dtype_code(h.dtype), _ptr(gu), M, inner, K, _stream(a))
    _check("fp8_block_grouped_gated_gemm", st)
    return h if gu is None else (h, gu)


def fp8_block_grouped_gated_gemm_quant(a, sa, offsets, w, sw, row_index=None, accum="fp8", pow2=False, q=None,
                                       scales=None, gu=None, save=False, workspace=None, stream=None):
    """The same with h leaving 1x128-quantised: ``(q, scales)``, and ``gu`` with ``save=True``."""
    if stream is not None:
        return _on_stream(stream, fp8_block_grouped_gated_gemm_quant, locals())
    if _elsewhere(a, sa, offsets, w, sw, row_index, q, scales, gu, workspace):
        return _over_there(a, fp8_block_grouped_gated_gemm_quant, locals())
    M = _segments(a, offsets, w, row_index)
    K, inner = _gated_operands(a, sa, w, sw, experts=True)
    q, gu = _gated_outputs(M, inner, torch.uint8, a, q, gu, save)
    scales = _scales_out(M, inner, a, scales)
    mode = _accum_code(accum, torch.bfloat16)
    L = _lib or lib()
    ws, nbytes = _workspace(L.fp8_block_gated_gemm_quant_workspace(mode, M, inner, K, w.shape[0]), workspace,
                            a.device)
    st = L.fp8_block_grouped_gated_gemm_quant(
        _ptr(a), _ptr(sa), a.shape[0], _ptr(row_index), _ptr(offsets), w.shape[0], _ptr(w), _ptr(sw), mode,
        1 if pow2 else 0, _ptr(q), _ptr(scales), _ptr(gu), _ptr(ws), nbytes, M, inner, K, _stream(a))
    _check("fp8_block_grouped_gated_gemm_quant", st)
    return (q, scales) if gu is None else (q, scales, gu)


def fp8_gated_backward_quant(dh, gu, pow2=False, rows=True, columns=True, h_columns=True, stream=None):
    """Gradient of the gated activation for ``dh`` [M, I] and the saved ``gu`` [M, 2I],
    quantised as it is formed.  Returns ``(q, s, q_t, s_t, q_ht, s_ht)``:

    ``rows``       q [M, 2I], s [M, 2I/128]: (dg, du), for the data gradient;
    ``columns``    q_t [2I, M], s_t [2I, M/128]: transposed, for the weight gradient;
    ``h_columns``  q_ht [I, M], s_ht [I, M/128]: h transposed, for the down
                   projection's weight gradient.
    A pair that is not asked for is (None, None)."""
    if stream is not None:
        return _on_stream(stream, fp8_gated_backward_quant, locals())
    if _elsewhere(dh, gu):
        return _over_there(dh, fp8_gated_backward_quant, locals())
    _rows(dh)
    _contig(gu)
    M, inner = dh.shape
    _like("gu", dh.dtype, (M, 2 * inner), gu)
    if (columns or h_columns) and M % 128 != 0:  # (fewer than 128 tokens would allocate scales of no columns)
        raise binding.Fp8fgError("fp8_gated_backward_quant", binding.ERR_UNSUPPORTED)

    def pair(want, n, k):
        if not want:
            return None, None
        return (torch.empty((n, k), dtype=torch.uint8, device=dh.device),
                torch.empty((n, k // 128), dtype=torch.float32, device=dh.device))

    out = (*pair(rows, M, 2 * inner), *pair(columns, 2 * inner, M), *pair(h_columns, inner, M))
    st = (_lib or lib()).fp8_gated_backward_quant(
        _ptr(dh), _ptr(gu), _dtype_code(dh.dtype), M, inner, _ld(dh), 1 if pow2 else 0, *[_ptr(t) for t in out],
        _stream(dh))
    _check("fp8_gated_backward_quant", st)
    return out


def _gradients(grads):
    """(device pointers, counts, type codes) of a list of gradients, as host arrays."""
    if False in [g.is_contiguous() for g in grads]:
        raise ValueError("gradients and outputs must be contiguous")
    codes = {d: _dtype_code(d) for d in {g.dtype for g in grads}}
    return (array("Q", [g.data_ptr() for g in grads]), array("q", [g.numel() for g in grads]),
            array("i", [codes[g.dtype] for g in grads]))


def _grad_norm(grads, outs, max_norm, norm, workspace):
    n = len(grads)
    tensors = [*grads, *(() if outs is None or outs is grads else outs),
               *(t for t in (norm, workspace) if t is not None)]
    if tensors and _elsewhere(*tensors):
        return _over_there(tensors[0], _grad_norm, dict(grads=grads, outs=outs, max_norm=max_norm, norm=norm,
                                                        workspace=workspace))
    ptrs, counts, dtypes = _gradients(grads)
    optrs = ptrs
    if outs is not None and outs is not grads:
        optrs, ocounts, odtypes = _gradients(outs)
        if ocounts != counts or odtypes != dtypes:
            raise ValueError("out must hold one tensor of the same type and length per gradient")
    dev = grads[0].device if n else torch.device("cuda", torch.cuda.current_device())
    if norm is None:
        norm = torch.empty((), dtype=torch.float32, device=dev)
    elif norm.dtype != torch.float32 or norm.numel() != 1:
        raise ValueError("norm must be one fp32 value")
    L = _lib or lib()
    ws, nbytes = _workspace(L.fp8fg_grad_norm_workspace(n), workspace, dev)
    host = [a.buffer_info()[0] for a in (ptrs, optrs, counts, dtypes)]  # (read during the call only)
    if outs is None:
        st = L.fp8fg_grad_norm(host[0], host[2], host[3], n, norm.data_ptr(), _ptr(ws), nbytes, _stream(norm))
        _check("fp8fg_grad_norm", st)
    else:
        st = L.fp8fg_clip_grad_norm(host[0], host[1], host[2], host[3], n, max_norm, norm.data_ptr(), _ptr(ws), nbytes,
                                    _stream(norm))
        _check("fp8fg_clip_grad_norm", st)
    return norm


def grad_norm(grads, norm=None, workspace=None, stream=None):
    """Global 2-norm over the list ``grads`` (fp32 or bf16, any lengths): an fp32 scalar on the device."""
    if stream is not None:
        return _on_stream(stream, grad_norm, locals())
    return _grad_norm(list(grads), None, 0.0, norm, workspace)


def clip_grad_norm(grads, max_norm, out=None, norm=None, workspace=None, stream=None):
    """Scale every tensor of ``grads`` by min(1, max_norm / norm), norm the global 2-norm.

    In place, or into the tensors of ``out`` (same types and lengths).  No tensor that is
    written may be listed twice, or overlap another of either list.  Returns the
    norm before clipping, an fp32 scalar on the device: no value comes back to the host."""
    if stream is not None:
        return _on_stream(stream, clip_grad_norm, locals())
    grads = list(grads)
    return _grad_norm(grads, grads if out is None else list(out), max_norm, norm, workspace)

"""ctypes binding of the layer operators of libfp8fg.so (include/fp8fg_layer.h).

The operators between the FP8 GEMMs of a feed-forward sublayer, with the same
names and the same rules as :mod:`fp8_fine_grained_amd.binding`: torch tensors
are device memory, outputs are allocated when none are given, every step runs
in the library's HIP kernels on torch's current stream (or ``stream=``), there
is no fallback, and a refused call raises :class:`binding.Fp8fgError`.
"""

import ctypes
import os

import torch

from . import binding
from .binding import _check, _contig, _dtype_code, _on_gpu, _ptr, _stream

HEADER = os.path.join(os.path.dirname(binding.HEADER), "fp8fg_layer.h")

_c = ctypes
_p, _i, _l, _f = _c.c_void_p, _c.c_int, _c.c_int64, _c.c_float
_SIGS = {
    "fp8_add_rmsnorm_quant_1x128": ([_p, _p, _i, _l, _l, _l, _l, _p, _i, _f, _i, _p, _p, _p, _p, _p, _p], _i),
    "fp8_rmsnorm_backward": ([_p, _p, _p, _i, _l, _l, _l, _l, _l, _p, _p, _i, _p, _p, _p, _l, _p], _i),
    "fp8_rmsnorm_backward_workspace": ([_l, _l], _l),
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


def _workspace(nbytes, given, device, stream):
    """``given``, or ``nbytes`` of fresh scratch memory.

    Fresh scratch is dropped when the call returns, before its kernels have run;
    the allocator reuses it only after the work of the current stream, so a call
    on another stream has to be made known to it."""
    if given is not None:
        _on_gpu(given)
        _contig(given)
        return given, given.numel() * given.element_size()
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    if stream is not None:
        s = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream), device=device)
        ws.record_stream(s)
    return ws, nbytes


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
        if t is not None and (t.dtype != dtype or tuple(t.shape) != tuple(shape)):
            raise ValueError(f"{what} must be {dtype} {list(shape)}")


def fp8_add_rmsnorm_quant_1x128(x, weight, residual=None, eps=1e-6, pow2=False, h=None, y=None, q=None, scales=None,
                                rstd=None, stream=None):
    """Residual addition, RMS norm and 1x128 quantisation of ``x`` [M, H] in one pass.

    ``x`` and ``residual`` are row-contiguous (any row pitch of whole 16 bytes).
    Pass ``y`` (of x's type) to also have the normed rows in high precision.
    Returns ``(h, q uint8 [M, H], scales fp32 [M, H/128], rstd fp32 [M])``;
    ``h`` is x + residual rounded to x's type, and x itself without a residual."""
    _on_gpu(x, weight, residual, h, y, q, scales, rstd)
    _rows(x, residual)
    M, H = x.shape
    _like("residual, h and y", x.dtype, (M, H), residual, h, y)
    if weight.dim() != 1 or weight.numel() != H or not weight.is_contiguous():
        raise ValueError("weight must be contiguous [H]")
    dev = x.device
    if residual is not None and h is None:
        h = torch.empty((M, H), dtype=x.dtype, device=dev)
    q = torch.empty((M, H), dtype=torch.uint8, device=dev) if q is None else q
    scales = torch.empty((M, H // 128), dtype=torch.float32, device=dev) if scales is None else scales
    rstd = torch.empty(M, dtype=torch.float32, device=dev) if rstd is None else rstd
    _like("q", torch.uint8, (M, H), q)
    _like("scales", torch.float32, (M, H // 128), scales)
    _like("rstd", torch.float32, (M,), rstd)
    _contig(*[t for t in (h, y, q, scales, rstd) if t is not None])
    st = lib().fp8_add_rmsnorm_quant_1x128(
        _ptr(x), _ptr(residual), _dtype_code(x.dtype), M, H, _ld(x), _ld(residual), _ptr(weight),
        _dtype_code(weight.dtype), eps, 1 if pow2 else 0, _ptr(h), _ptr(y), _ptr(q), _ptr(scales), _ptr(rstd),
        _stream(stream))
    _check("fp8_add_rmsnorm_quant_1x128", st)
    return x if h is None else h, q, scales, rstd


def fp8_rmsnorm_backward(dy, h, rstd, weight, dh=None, dx=None, dw=None, need_dw=True, workspace=None, stream=None):
    """Gradient of the norm: ``(dx [M, H] of dy's type, dw fp32 [H])``.

    ``h`` and ``rstd`` as the forward call returned them; ``dh`` is the gradient
    that arrives along the residual stream.  ``need_dw=False``: dw is None."""
    _on_gpu(dy, h, rstd, weight, dh, dx, dw)
    _rows(dy, h, dh)
    M, H = dy.shape
    _like("h, dh and dx", dy.dtype, (M, H), h, dh, dx)
    _like("rstd", torch.float32, (M,), rstd)
    _like("dw", torch.float32, (H,), dw)
    if weight.dim() != 1 or weight.numel() != H:
        raise ValueError("weight must be [H]")
    dx = torch.empty((M, H), dtype=dy.dtype, device=dy.device) if dx is None else dx
    if dw is None and need_dw:
        dw = torch.empty(H, dtype=torch.float32, device=dy.device)
    _contig(rstd, weight, dx, *([dw] if dw is not None else []))
    ws, nbytes = None, 0
    if dw is not None:
        ws, nbytes = _workspace(lib().fp8_rmsnorm_backward_workspace(M, H), workspace, dy.device, stream)
    st = lib().fp8_rmsnorm_backward(
        _ptr(dy), _ptr(h), _ptr(dh), _dtype_code(dy.dtype), M, H, _ld(dy), _ld(h), _ld(dh), _ptr(rstd), _ptr(weight),
        _dtype_code(weight.dtype), _ptr(dx), _ptr(dw), _ptr(ws), nbytes, _stream(stream))
    _check("fp8_rmsnorm_backward", st)
    return dx, dw


def _grad_arrays(grads):
    n = len(grads)
    for g in grads:
        if not g.is_cuda:
            raise ValueError("all tensors must be on the GPU")
        if not g.is_contiguous():
            raise ValueError("gradients and outputs must be contiguous")
    return ((_c.c_void_p * n)(*[g.data_ptr() for g in grads]), (_c.c_int64 * n)(*[g.numel() for g in grads]),
            (_c.c_int * n)(*[_dtype_code(g.dtype) for g in grads]))


def grad_norm(grads, norm=None, workspace=None, stream=None):
    """Global 2-norm over the list ``grads`` (fp32 or bf16, any lengths): an fp32 scalar on the device."""
    grads = list(grads)
    ptrs, counts, dtypes = _grad_arrays(grads)
    dev = grads[0].device if grads else torch.device("cuda")
    norm = torch.empty((), dtype=torch.float32, device=dev) if norm is None else norm
    ws, nbytes = _workspace(lib().fp8fg_grad_norm_workspace(len(grads)), workspace, dev, stream)
    st = lib().fp8fg_grad_norm(ptrs, counts, dtypes, len(grads), _ptr(norm), _ptr(ws), nbytes, _stream(stream))
    _check("fp8fg_grad_norm", st)
    return norm


def clip_grad_norm(grads, max_norm, out=None, norm=None, workspace=None, stream=None):
    """Scale every tensor of ``grads`` by min(1, max_norm / norm), norm the global 2-norm.

    In place, or into the tensors of ``out`` (same types and lengths).  Returns the
    norm before clipping, an fp32 scalar on the device: no value comes back to the host."""
    grads = list(grads)
    outs = grads if out is None else list(out)
    if len(outs) != len(grads) or any(o.dtype != g.dtype or o.numel() != g.numel() for o, g in zip(outs, grads)):
        raise ValueError("out must hold one tensor of the same type and length per gradient")
    ptrs, counts, dtypes = _grad_arrays(grads)
    optrs = ptrs if out is None else _grad_arrays(outs)[0]
    dev = grads[0].device if grads else torch.device("cuda")
    norm = torch.empty((), dtype=torch.float32, device=dev) if norm is None else norm
    ws, nbytes = _workspace(lib().fp8fg_grad_norm_workspace(len(grads)), workspace, dev, stream)
    st = lib().fp8fg_clip_grad_norm(ptrs, optrs, counts, dtypes, len(grads), max_norm, _ptr(norm), _ptr(ws), nbytes,
                                    _stream(stream))
    _check("fp8fg_clip_grad_norm", st)
    return norm

"""What stands around a linear layer in training, on torch tensors: the layer norm
with its gradient, and the norm and clipping of a network's gradients, over the C
entry points of include/swz.h (argument marshalling only; every computation runs
in the library's kernels).

All operands of a call are on the current device; ``stream`` is as in ``linear``.
``layer_norm`` is the form with a gradient; ``layer_norm_forward`` and
``_backward`` are for callers who carry gradients themselves.
"""
from __future__ import annotations

import ctypes
import math
from array import array

import thread_block_smem_gb300 as _swz

from . import linear as _lin


class swz_grad(ctypes.Structure):
    _fields_ = [("in_", ctypes.c_void_p), ("out", ctypes.c_void_p), ("n", ctypes.c_int64),
                ("dtype", ctypes.c_int), ("out_dtype", ctypes.c_int)]


def declare(L):
    """Argument types of this module's entry points on the loaded library."""
    i, i64, u64, vp, f = (ctypes.c_int, ctypes.c_int64, ctypes.c_uint64, ctypes.c_void_p,
                          ctypes.c_double)
    L.swz_layer_norm.argtypes = [vp, i, i64, vp, i, vp, i, f, vp, i, i64, vp, vp, i, i, vp]
    L.swz_layer_norm_backward.argtypes = [vp, i, i64, vp, i, i64, vp, i, vp, vp, vp, i, i64, vp, vp,
                                          i, i, i, vp, u64, vp]
    L.swz_layer_norm_backward_workspace_size.argtypes = [i, i, ctypes.POINTER(u64)]
    L.swz_grad_norm.argtypes = [vp, i, vp, vp, u64, vp]
    L.swz_clip_grad_norm.argtypes = [vp, i, f, f, vp, vp, u64, vp]
    L.swz_grad_norm_workspace_size.argtypes = [i, ctypes.POINTER(u64)]


# ---- raw mirrors ----------------------------------------------------------------
def swz_layer_norm(x, dtype, ldx, weight, w_dtype, bias, b_dtype, eps, y, y_dtype, ldy, mean, rstd,
                   M, N, stream=0):
    if not _lin._ints(dtype, w_dtype, b_dtype, y_dtype, M, N):
        return _swz.SWZ_EINVAL
    return _swz.lib().swz_layer_norm(x, dtype, ldx, weight, w_dtype, bias, b_dtype, eps, y, y_dtype,
                                     ldy, mean, rstd, M, N, stream)


def swz_layer_norm_backward(dy, dy_dtype, lddy, x, dtype, ldx, weight, w_dtype, mean, rstd, dx,
                            dx_dtype, lddx, dw, db, dw_dtype, M, N, workspace, workspace_bytes,
                            stream=0):
    if not _lin._ints(dy_dtype, dtype, w_dtype, dx_dtype, dw_dtype, M, N):
        return _swz.SWZ_EINVAL
    return _swz.lib().swz_layer_norm_backward(dy, dy_dtype, lddy, x, dtype, ldx, weight, w_dtype,
                                              mean, rstd, dx, dx_dtype, lddx, dw, db, dw_dtype, M, N,
                                              workspace, workspace_bytes, stream)


def swz_layer_norm_backward_workspace_size(M, N):
    if not _lin._ints(M, N):
        return _swz.SWZ_EINVAL, 0
    b = ctypes.c_uint64(0)
    rc = _swz.lib().swz_layer_norm_backward_workspace_size(M, N, ctypes.byref(b))
    return rc, b.value


def swz_grad_norm(grads, count, norm, workspace, workspace_bytes, stream=0):
    if not _lin._ints(count):
        return _swz.SWZ_EINVAL
    return _swz.lib().swz_grad_norm(grads, count, norm, workspace, workspace_bytes, stream)


def swz_clip_grad_norm(grads, count, max_norm, eps, norm, workspace, workspace_bytes, stream=0):
    if not _lin._ints(count):
        return _swz.SWZ_EINVAL
    return _swz.lib().swz_clip_grad_norm(grads, count, max_norm, eps, norm, workspace,
                                         workspace_bytes, stream)


def swz_grad_norm_workspace_size(count):
    if not _lin._ints(count):
        return _swz.SWZ_EINVAL, 0
    b = ctypes.c_uint64(0)
    rc = _swz.lib().swz_grad_norm_workspace_size(count, ctypes.byref(b))
    return rc, b.value


# ---- layer norm -------------------------------------------------------------------
def _vector(v, n, what):
    """(address, type code) of a weight or bias of n values; None: (None, any code)."""
    if v is None:
        return None, _lin.SWZ_F32
    if v.dim() != 1 or v.shape[0] != n:
        raise ValueError(f"{what}: shape {(n,)} expected, got {tuple(v.shape)}")
    if n > 1 and v.stride(0) != 1:
        raise ValueError(f"{what}: contiguous values expected")
    return v.data_ptr(), _lin._code(v.dtype, what)


def _statistic(v, m, what):
    """Address of the mean or rstd of m rows."""
    if v.dtype != _lin.torch.float32:
        raise TypeError(f"{what}: fp32 expected")
    if v.dim() != 1 or v.shape[0] != m or (m > 1 and v.stride(0) != 1):
        raise ValueError(f"{what}: {m} contiguous values expected")
    return v.data_ptr()


def layer_norm_forward(x, weight=None, bias=None, eps=1e-5, *, out=None, out_dtype=None,
                       stream=None):
    """(y, mean, rstd) of the rows of x (M x N; fp16, bf16 or fp32, contiguous rows):
    y = (x - mean) rstd weight + bias, rstd = 1 / sqrt(var + eps) with the mean square
    of x - mean as var.  ``weight`` and ``bias`` (N values, of any of the types) may be
    None.  ``out`` (M x N; may be x itself, refused where it lies across an operand) or
    ``out_dtype`` (default: x's type).  mean and rstd (fp32) are for
    layer_norm_backward."""
    if _lin.torch is None:
        _lin._init()
    torch = _lin.torch
    _lin._here(x, weight, bias, out)
    M, N, ldx = _lin._rows(x, "x")
    code = _lin._code(x.dtype, "x")
    pw, wcode = _vector(weight, N, "weight")
    pb, bcode = _vector(bias, N, "bias")
    y, ldy, ycode = _lin._output(out, out_dtype or x.dtype, M, N, x, stream)
    if stream is not None:
        _lin._keep(stream, x, weight, bias, out)
    mean = _lin._empty(M, torch.float32, x, stream)
    rstd = _lin._empty(M, torch.float32, x, stream)
    rc = _lin._L.swz_layer_norm(x.data_ptr(), code, ldx, pw, wcode, pb, bcode, eps, y.data_ptr(),
                                ycode, ldy, mean.data_ptr(), rstd.data_ptr(), M, N,
                                _lin._handle(stream, x))
    if rc:
        raise _swz.SwzError(rc, "swz_layer_norm")
    if out is not None:
        _swz._written(out)
    return y, mean, rstd


def layer_norm_backward(dy, x, weight, mean, rstd, *, need_dx=True, need_dw=True, need_db=True,
                        dx_dtype=None, dw_dtype=None, stream=None):
    """(dx, dw, db) of layer_norm_forward: dx (M x N; default x's type), dw and db (N
    values; default fp32); None in place of one that is not needed.  With g = dy weight
    and xhat = (x - mean) rstd: dx = rstd (g - mean(g) - xhat mean(g xhat)), dw the sum
    of dy xhat over the rows, db that of dy."""
    if _lin.torch is None:
        _lin._init()
    torch = _lin.torch
    _lin._here(dy, x, weight, mean, rstd)
    M, N, lddy = _lin._rows(dy, "dy")
    Mx, Nx, ldx = _lin._rows(x, "x")
    if (Mx, Nx) != (M, N):
        raise ValueError("dy does not have the shape of x")
    ycode, code = _lin._code(dy.dtype, "dy"), _lin._code(x.dtype, "x")
    pw, wcode = _vector(weight, N, "weight")
    pm, pr = _statistic(mean, M, "mean"), _statistic(rstd, M, "rstd")
    if stream is not None:
        _lin._keep(stream, dy, x, weight, mean, rstd)
    if not (need_dx or need_dw or need_db):
        return None, None, None
    dx_dtype, dw_dtype = dx_dtype or x.dtype, dw_dtype or torch.float32
    xcode, gcode = _lin._code(dx_dtype, "dx_dtype"), _lin._code(dw_dtype, "dw_dtype")
    dx = _lin._empty((M, N), dx_dtype, x, stream) if need_dx else None
    dw = _lin._empty(N, dw_dtype, x, stream) if need_dw else None
    db = _lin._empty(N, dw_dtype, x, stream) if need_db else None
    ws, need = None, 0
    if need_dw or need_db:
        rc, need = swz_layer_norm_backward_workspace_size(M, N)
        _swz._check(rc, "swz_layer_norm_backward_workspace_size")
        ws = _lin._empty(need, torch.uint8, x, stream)
    rc = _lin._L.swz_layer_norm_backward(
        dy.data_ptr(), ycode, lddy, x.data_ptr(), code, ldx, pw, wcode, pm, pr,
        dx.data_ptr() if need_dx else None, xcode, N, dw.data_ptr() if need_dw else None,
        db.data_ptr() if need_db else None, gcode, M, N, ws.data_ptr() if need else None, need,
        _lin._handle(stream, x))
    if rc:
        raise _swz.SwzError(rc, "swz_layer_norm_backward")
    return dx, dw, db


_function = None


def layer_norm(x, weight=None, bias=None, eps=1e-5):
    """y = (x - mean) rstd weight + bias over the last dimension of x (..., N), with its
    gradient for torch.autograd; x of any layout (copied where rows are not contiguous),
    y of x's type.  The gradients of weight and bias are summed in fp32 and rounded to
    their types.  A second derivative raises."""
    global _function
    if _function is None:
        if _lin.torch is None:
            _lin._init()
        torch = _lin.torch

        class LayerNorm(torch.autograd.Function):
            @staticmethod
            def forward(ctx, x, weight, bias, eps):
                x = _lin._with_rows(x)
                y, mean, rstd = layer_norm_forward(x, weight, bias, eps)
                ctx.save_for_backward(x, weight, mean, rstd)
                ctx.bias_dtype = None if bias is None else bias.dtype
                return y

            @staticmethod
            @torch.autograd.function.once_differentiable
            def backward(ctx, dy):
                x, weight, mean, rstd = ctx.saved_tensors
                need_dx, need_dw, need_db = ctx.needs_input_grad[:3]
                types = {t for t, need in ((weight.dtype if need_dw else None, need_dw),
                                           (ctx.bias_dtype, need_db)) if need}
                dx, dw, db = layer_norm_backward(
                    _lin._with_rows(dy), x, weight, mean, rstd, need_dx=need_dx, need_dw=need_dw,
                    need_db=need_db, dw_dtype=types.pop() if len(types) == 1 else None)
                return (dx, dw if dw is None else dw.to(weight.dtype),
                        db if db is None else db.to(ctx.bias_dtype), None)

        _function = LayerNorm
    flat = x.reshape(math.prod(x.shape[:-1]), x.shape[-1])
    return _function.apply(flat, weight, bias, eps).reshape(x.shape)


# ---- gradients of a network ---------------------------------------------------------
def _dense(t):
    """Whether t's values fill one piece of memory, in any order of its dimensions."""
    n = 1
    for size, stride in sorted(zip(t.shape, t.stride()), key=lambda d: d[1]):
        if size == 1:
            continue
        if stride != n:
            return False
        n *= size
    return True


def _grads(grads, out, stream):
    """(array of swz_grad records, count, a tensor of the list) of checked gradients."""
    torch = _lin.torch
    if not grads:
        raise ValueError("grads: one tensor at least expected")
    codes = _lin._codes
    dev = grads[0].get_device()
    _lin._here(grads[0])
    records = array("Q")
    for i, g in enumerate(grads):
        o = g if out is None else out[i]
        code, ocode = codes.get(g.dtype), codes.get(o.dtype)
        if code is None or ocode is None:
            raise TypeError("gradients must be fp16, bf16 or fp32")
        if g.get_device() != dev or o.get_device() != dev:
            raise ValueError("operands are on different devices")
        if not g.is_contiguous() and not _dense(g):
            raise ValueError("gradients must fill one piece of memory each")
        if o is not g:
            if o.shape != g.shape:
                raise ValueError(f"out: shape {tuple(g.shape)} expected")
            if o.stride() != g.stride() and not (o.is_contiguous() and g.is_contiguous()):
                raise ValueError("out: the gradient's strides expected")
        if (g.requires_grad or o.requires_grad) and torch.is_grad_enabled():
            raise ValueError("grad_norm and clip_grad_norm have no gradient: tensors that "
                             "require one are refused")
        records.extend((g.data_ptr(), o.data_ptr(), g.numel(), code | ocode << 32))
    if stream is not None:
        _lin._keep(stream, *grads, *(out or ()))
    return records


def _norm_call(name, grads, out, stream, *limits):
    torch = _lin.torch
    records = _grads(grads, out, stream)
    norm = _lin._empty((), torch.float32, grads[0], stream)
    rc, need = swz_grad_norm_workspace_size(len(grads))
    _swz._check(rc, "swz_grad_norm_workspace_size")
    ws = _lin._empty(need, torch.uint8, grads[0], stream)
    rc = getattr(_lin._L, name)(records.buffer_info()[0], len(grads), *limits, norm.data_ptr(),
                                ws.data_ptr(), need, _lin._handle(stream, grads[0]))
    if rc:
        raise _swz.SwzError(rc, name)
    return norm


def grad_norm(grads, *, stream=None):
    """The norm of all gradients together (a scalar fp32 tensor on the device): the
    square root of the sum of their squares.  ``grads``: tensors of any shapes, fp16,
    bf16 or fp32 each, that fill one piece of memory each."""
    if _lin.torch is None:
        _lin._init()
    return _norm_call("swz_grad_norm", list(grads), None, stream)


def clip_grad_norm(grads, max_norm, eps=1e-6, *, out=None, stream=None):
    """Multiplies all gradients by min(1, max_norm / (norm + eps)) in place, or writes
    the products to the tensors of ``out`` (the same shapes, and the same strides where
    the gradients' own are not contiguous; fp16, bf16 or fp32 each),
    and returns the norm they had, a scalar fp32 tensor on the device, without waiting
    for it.  ``grads`` as in ``grad_norm``; no result may lie over another tensor.  A NaN
    among the gradients makes all of them NaN; an infinity makes the finite ones zero."""
    if _lin.torch is None:
        _lin._init()
    grads = list(grads)
    if out is not None:
        out = list(out)
        if len(out) != len(grads):
            raise ValueError("out: one tensor for each gradient expected")
    max_norm, eps = float(max_norm), float(eps)
    if not max_norm >= 0 or not eps >= 0:
        raise ValueError("max_norm and eps must be at least 0")
    norm = _norm_call("swz_clip_grad_norm", grads, out, stream, max_norm, eps)
    _swz._written(*(grads if out is None else out))
    return norm

"""Linear layers in 8 bits on torch tensors: block quantisation, the product of
8-bit operands, the layer's forward and gradient, over the C entry points of
include/swz.h (argument marshalling only; every computation runs in the
library's kernels).

8-bit matrices are ``torch.float8_e4m3fn`` or ``torch.float8_e5m2`` tensors of
shape (rows, K) whose rows start on multiples of 16 bytes (``quantize_fp8``
makes them so; ``fp8_empty`` allocates one).  Scales are fp32: of ``"row"``
blocks (1 x 128) a tensor (ceil(K / 128), rows), of ``"square"`` ones (128 x
128) a tensor (ceil(rows / 128), ceil(K / 128)).  All operands of a call are on
the current device.  ``stream`` (a torch stream, or a cudaStream_t as an int) is
what a call runs on instead of the current one; its operands may be freed while a
torch stream still works on them, and what it returns belongs to that stream.

``fp8_linear`` is the form with a gradient.  ``gemm_fp8``, ``linear_fp8`` and
``newton_schulz`` have none: a backward through what they return raises
(``out`` takes values only), and ``linear_fp8_forward`` and ``_backward`` are for
callers who carry gradients themselves.
"""
from __future__ import annotations

import contextlib
import ctypes
import math

import thread_block_smem_gb300 as _swz

SWZ_F32 = 3
SWZ_E4M3, SWZ_E5M2 = 0, 1
SWZ_BLOCK_ROW, SWZ_BLOCK_SQUARE = 0, 1
BLOCK = 128
BLOCKS = {"row": SWZ_BLOCK_ROW, "square": SWZ_BLOCK_SQUARE}
FORMATS = {"e4m3": SWZ_E4M3, "e5m2": SWZ_E5M2}


class swz_fp8_matrix(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("ld", ctypes.c_int64), ("scales", ctypes.c_void_p),
                ("ld_scales", ctypes.c_int64), ("fmt", ctypes.c_int), ("block", ctypes.c_int)]


class swz_gemm_fp8_opts(ctypes.Structure):
    _fields_ = [("order", ctypes.c_int), ("group", ctypes.c_int), ("tile", ctypes.c_int),
                ("split_k", ctypes.c_int), ("num_programs", ctypes.c_int),
                ("debug_flags", ctypes.c_uint32), ("timeout_ms", ctypes.c_uint32)]


class swz_newton_schulz_opts(ctypes.Structure):
    _fields_ = [("tile", ctypes.c_int), ("debug_flags", ctypes.c_uint32),
                ("timeout_ms", ctypes.c_uint32)]


def declare(L):
    """Argument types of this module's entry points on the loaded library."""
    i, i64, u64, vp = ctypes.c_int, ctypes.c_int64, ctypes.c_uint64, ctypes.c_void_p
    mat = ctypes.POINTER(swz_fp8_matrix)
    L.swz_quantize_fp8.argtypes = [vp, i, i64, i, i, i, i, vp, i64, vp, i64, vp, i64, vp, i64, vp]
    L.swz_gemm_fp8.argtypes = [mat, mat, vp, i64, i, i, i, i, ctypes.POINTER(swz_gemm_fp8_opts), vp]
    L.swz_linear_fp8.argtypes = [vp, i, i64, mat, vp, i64, i, i, i, i, vp, u64, vp]
    L.swz_linear_fp8_workspace_size.argtypes = [i, i, i, ctypes.POINTER(u64)]
    f = ctypes.c_double
    L.swz_newton_schulz.argtypes = [vp, i, i64, i64, vp, i, i64, i64, i, i, i, i, f, f, f, f,
                                    ctypes.POINTER(swz_newton_schulz_opts), vp, u64, vp]
    L.swz_newton_schulz_workspace_size.argtypes = [i, i, i, ctypes.POINTER(u64)]


# ---- raw mirrors ----------------------------------------------------------------
# ctypes hands a C int the low 32 bits of a larger number without a word, so the
# mirrors refuse what does not fit as the entry points refuse other sizes.
INT_MAX = 2 ** 31 - 1


def _ints(*values):
    """True when every value fits a C int."""
    return all(-INT_MAX <= v <= INT_MAX for v in values)


def swz_quantize_fp8(x, dtype, ldx, M, K, block, fmt, q, ldq, scales, ld_scales, qt, ldqt,
                     scales_t, ld_scales_t, stream=0):
    if not _ints(dtype, M, K, block, fmt):
        return _swz.SWZ_EINVAL
    return _swz.lib().swz_quantize_fp8(x, dtype, ldx, M, K, block, fmt, q, ldq, scales, ld_scales,
                                       qt, ldqt, scales_t, ld_scales_t, stream)


def swz_gemm_fp8(A, B, C, ldc, c_dtype, M, N, K, opts=None, stream=0):
    if not _ints(c_dtype, M, N, K):
        return _swz.SWZ_EINVAL
    return _swz.lib().swz_gemm_fp8(ctypes.byref(A), ctypes.byref(B), C, ldc, c_dtype, M, N, K,
                                   ctypes.byref(opts) if opts is not None else None, stream)


def swz_linear_fp8(x, dtype, ldx, W, y, ldy, y_dtype, M, N, K, workspace, workspace_bytes,
                   stream=0):
    if not _ints(dtype, y_dtype, M, N, K):
        return _swz.SWZ_EINVAL
    return _swz.lib().swz_linear_fp8(x, dtype, ldx, ctypes.byref(W), y, ldy, y_dtype, M, N, K,
                                     workspace, workspace_bytes, stream)


def swz_linear_fp8_workspace_size(M, N, K):
    if not _ints(M, N, K):
        return _swz.SWZ_EINVAL, 0
    b = ctypes.c_uint64(0)
    rc = _swz.lib().swz_linear_fp8_workspace_size(M, N, K, ctypes.byref(b))
    return rc, b.value


def swz_newton_schulz(G, dtype, ldg, batch_stride_g, Y, y_dtype, ldy, batch_stride_y, batch, m, n,
                      steps, a, b, c, eps, opts, workspace, workspace_bytes, stream=0):
    if not _ints(dtype, y_dtype, batch, m, n, steps):
        return _swz.SWZ_EINVAL
    return _swz.lib().swz_newton_schulz(
        G, dtype, ldg, batch_stride_g, Y, y_dtype, ldy, batch_stride_y, batch, m, n, steps, a, b,
        c, eps, ctypes.byref(opts) if opts is not None else None, workspace, workspace_bytes,
        stream)


def swz_newton_schulz_workspace_size(batch, m, n):
    if not _ints(batch, m, n):
        return _swz.SWZ_EINVAL, 0
    b = ctypes.c_uint64(0)
    rc = _swz.lib().swz_newton_schulz_workspace_size(batch, m, n, ctypes.byref(b))
    return rc, b.value


# ---- helpers ----------------------------------------------------------------------
# A call on small tensors costs the host more than the GPU, so what every call
# needs is looked up once: torch, the type codes, the library.
torch = None
_u64 = ctypes.c_uint64
_codes = _f8_codes = _f8_types = _L = _NoGradient = None


def _init():
    global torch, _codes, _f8_codes, _f8_types, _L, _NoGradient
    import torch as t
    _codes = {t.float16: _swz.SWZ_F16, t.bfloat16: _swz.SWZ_BF16, t.float32: SWZ_F32}
    _f8_codes = {t.float8_e4m3fn: SWZ_E4M3, t.float8_e5m2: SWZ_E5M2}
    _f8_types = {"e4m3": t.float8_e4m3fn, "e5m2": t.float8_e5m2}
    _L = _swz.lib()

    class NoGradient(t.autograd.Function):
        @staticmethod
        def forward(ctx, what, y, *inputs):
            ctx.what = what
            ctx.mark_dirty(y)
            return y

        @staticmethod
        def backward(ctx, *dy):
            raise RuntimeError(f"{ctx.what} has no gradient (fp8_linear has one)")

    _NoGradient = NoGradient
    torch = t


def _code(t, what):
    code = _codes.get(t)
    if code is None:
        raise TypeError(f"{what} must be fp16, bf16 or fp32")
    return code


def _rows(x, what):
    """(rows, columns, elements from row to row) of a 2-D tensor with contiguous rows."""
    if x.dim() != 2:
        raise ValueError(f"{what}: 2-D tensor expected")
    if not x.is_cuda:
        raise ValueError(f"{what}: CUDA tensor expected")
    m, k = x.shape
    if (m | k) > INT_MAX:
        raise ValueError(f"{what}: more than 2^31 - 1 rows or columns")
    ld, one = x.stride()
    if one != 1 and k > 1 and m > 0:
        raise ValueError(f"{what}: contiguous rows expected")
    if m <= 1:
        return m, k, k or 1
    if ld < k:
        raise ValueError(f"{what}: rows must not overlap")
    return m, k, ld


def _in_range(debug_flags, timeout_ms, *ints):
    """Refuses options that their C types would cut."""
    if not (_ints(*ints) and 0 <= debug_flags < 2 ** 32 and 0 <= timeout_ms < 2 ** 32):
        raise ValueError("option out of range")


def _here(x, *others):
    """Refuses operands that are not all on the current device: the library
    launches there, and a default stream's handle does not say whose it is."""
    dev = x.get_device()
    for t in others:
        if t is not None and t.get_device() != dev:
            raise ValueError("operands are on different devices")
    if dev < 0:
        raise ValueError("CUDA tensors expected")
    if dev != torch._C._cuda_getDevice():
        raise ValueError(f"operands are on cuda:{dev}, which is not the current device")


def _on(stream):
    """Context in which what is allocated belongs to the stream that the call runs on."""
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream))
    return torch.cuda.stream(stream)


def _keep(stream, *tensors):
    """Memory of the operands that is freed is not handed out again before
    `stream` is done with them.  Only for streams of torch's own: others are their
    maker's, who may destroy them before the operands."""
    if (not isinstance(stream, torch.cuda.Stream) or
            isinstance(stream, torch.cuda.ExternalStream)):
        return
    for t in tensors:
        if t is not None:
            t.record_stream(stream)


def _handle(stream, x):
    """The cudaStream_t that a call runs on (None: the current stream of x's
    device, which _here has found to be the current one)."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(x.device.index)
    return _swz._stream(stream)


def _empty(shape, dtype, x, stream):
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=x.device)
    with _on(stream):
        return torch.empty(shape, dtype=dtype, device=x.device)


def _block(block):
    code = BLOCKS.get(block)
    if code is None:
        raise ValueError("block must be 'row' or 'square'")
    return code


def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


def fp8_empty(rows, cols, dtype, device="cuda"):
    """Uninitialised 8-bit (rows, cols) tensor whose rows start on multiples of 16 bytes."""
    if torch is None:
        _init()
    ld = (cols + 15) // 16 * 16
    q = torch.empty((rows, ld), dtype=dtype, device=device)
    return q if ld == cols else q.narrow(1, 0, cols)


def _matrix(q, scales, block, what):
    """swz_fp8_matrix of an 8-bit tensor and its scales, checked."""
    fmt = _f8_codes.get(q.dtype)
    if fmt is None:
        raise TypeError(f"{what}: float8_e4m3fn or float8_e5m2 expected")
    m, k, ld = _rows(q, what)
    if m <= 1 or k == 0:  # no second row whose place matters
        ld = (k + 15) // 16 * 16
    at = q.data_ptr()
    if ld % 16 or at % 16:
        raise ValueError(f"{what}: rows must start on multiples of 16 bytes")
    if scales.dtype != torch.float32 or not scales.is_cuda:
        raise TypeError(f"{what}: fp32 CUDA scales expected")
    want = (_blocks(k), m) if block == SWZ_BLOCK_ROW else (_blocks(m), _blocks(k))
    if scales.shape != want:
        raise ValueError(f"{what}: scales of shape {want} expected, got {tuple(scales.shape)}")
    _, _, lds = _rows(scales, what)
    return swz_fp8_matrix(at, ld, scales.data_ptr(), lds, fmt, block), m, k


def _output(out, dtype, M, N, x, stream):
    """(tensor, elements from row to row, type code) of an M x N result."""
    if out is None:
        code = _code(dtype, "out_dtype")
        return _empty((M, N), dtype, x, stream), N, code
    code = _code(out.dtype, "out")
    m, n, ld = _rows(out, "out")
    if m != M or n != N:
        raise ValueError(f"out: shape {(M, N)} expected")
    return out, ld, code


def _no_gradient(what, y, *inputs):
    """y, through which a backward raises if one of the inputs asks for a gradient:
    the library's kernels record none, and without this it would just be missing."""
    for t in inputs:
        if t.requires_grad and torch.is_grad_enabled():
            return _NoGradient.apply(what, y, *inputs)
    return y


def _result(what, y, out, *inputs):
    """What a call returns that has written y, which is ``out`` where that was given."""
    if out is None:
        return _no_gradient(what, y, *inputs)
    if isinstance(out, torch.Tensor):  # (what only looks like one has no version)
        _swz._written(out)
    return out


# ---- operators --------------------------------------------------------------------
def quantize_fp8(x, block="row", fmt="e4m3", transposed=False, *, stream=None):
    """(q, scales) of x (M x K; fp16, bf16 or fp32, contiguous rows), with
    ``transposed`` (q, scales, qt, scales_t): also x^T (K x M) in 8 bits, by
    blocks of its own rows or by the same squares, in the same read of x.

    For a block with largest magnitude amax: ac = max(amax, 2^-96), r = F / ac,
    scale = ac / F (F = 448 for e4m3, 57344 for e5m2), q = x r rounded to
    nearest even."""
    if torch is None:
        _init()
    _here(x)
    q, s, qt, st, M, K = _quantize(x, _block(block), fmt, transposed, stream)
    q = q if q.shape[1] == K else q.narrow(1, 0, K)
    if not transposed:
        return q, s
    return q, s, (qt if qt.shape[1] == M else qt.narrow(1, 0, M)), st


def _quantize(x, b, fmt, transposed, stream):
    """(q, scales, qt, scales_t, M, K), q and qt with whole rows of a multiple of 16 bytes."""
    M, K, ldx = _rows(x, "x")
    code, f = _code(x.dtype, "x"), FORMATS.get(fmt)
    if f is None:
        raise ValueError("fmt must be 'e4m3' or 'e5m2'")
    if stream is not None:
        _keep(stream, x)
    f8 = _f8_types[fmt]
    kb, mb = (K + 127) // 128, (M + 127) // 128
    ldq, ldt = (K + 15) // 16 * 16, (M + 15) // 16 * 16
    q = _empty((M, ldq), f8, x, stream)
    s = _empty((mb, kb) if b else (kb, M), torch.float32, x, stream)
    qt = st = None
    to = (None, 0, None, 0)
    if transposed:
        qt = _empty((K, ldt), f8, x, stream)
        st = _empty((kb, mb) if b else (mb, K), torch.float32, x, stream)
        to = (qt.data_ptr(), ldt, st.data_ptr(), mb if b else K)
    rc = _L.swz_quantize_fp8(x.data_ptr(), code, ldx, M, K, b, f, q.data_ptr(), ldq, s.data_ptr(),
                             kb if b else M, *to, _handle(stream, x))
    if rc:
        raise _swz.SwzError(rc, "swz_quantize_fp8")
    return q, s, qt, st, M, K


def _own(q, s, fmt, block):
    """swz_fp8_matrix of what _quantize made: nothing to check."""
    return swz_fp8_matrix(q.data_ptr(), q.shape[1], s.data_ptr(), s.shape[1], fmt, block)


def _product(A, B, M, N, K, dtype, x, stream):
    """C = A B^T (M x N of `dtype`) of checked operands, in the default order."""
    code = _code(dtype, "out_dtype")
    C = _empty((M, N), dtype, x, stream)
    rc = _L.swz_gemm_fp8(A, B, C.data_ptr(), N, code, M, N, K, None, _handle(stream, x))
    if rc:
        raise _swz.SwzError(rc, "swz_gemm_fp8")
    return C


def gemm_fp8(a, sa, b, sb, *, b_block="square", out=None, out_dtype=None, order="serpentine",
             group=8, tile=0, split_k=0, num_programs=0, debug_flags=0, timeout_ms=0,
             stream=None):
    """C = A B^T (M x N) of 8-bit operands: a (M x K) with scales sa of its row
    blocks, b (N x K) with scales sb of its ``b_block`` blocks.  ``out`` (M x
    N, contiguous rows) or ``out_dtype`` (fp32, bf16 or fp16; default bf16).
    ``order``, ``group``: the order of the output tiles, as in ``gemm``;
    ``tile``, ``split_k``, ``num_programs``: see swz_gemm_fp8_opts (0 =
    automatic)."""
    if torch is None:
        _init()
    _here(a, sa, b, sb, out)
    A, M, K = _matrix(a, sa, SWZ_BLOCK_ROW, "a")
    B, N, K2 = _matrix(b, sb, _block(b_block), "b")
    if K != K2:
        raise ValueError("inner dimensions differ")
    order = _swz._order(order)
    _in_range(debug_flags, timeout_ms, order, group, tile, split_k, num_programs)
    C, ldc, code = _output(out, out_dtype or torch.bfloat16, M, N, a, stream)
    if stream is not None:
        _keep(stream, a, sa, b, sb, out)
    opts = swz_gemm_fp8_opts(order, group, tile, split_k, num_programs, debug_flags,
                             timeout_ms)
    _swz._check(_L.swz_gemm_fp8(A, B, C.data_ptr(), ldc, code, M, N, K, opts, _handle(stream, a)),
                "swz_gemm_fp8")
    return _result("gemm_fp8", C, out, a, sa, b, sb)


def linear_fp8(x, qw, sw, *, w_block="square", out=None, out_dtype=None, stream=None):
    """y = x W^T (M x N): x (M x K; fp16, bf16 or fp32) is quantised in row
    blocks (e4m3) and multiplied by W (N x K) kept as (qw, sw).  ``out`` or
    ``out_dtype`` (default: x's type)."""
    if torch is None:
        _init()
    _here(x, qw, sw, out)
    M, K, ldx = _rows(x, "x")
    code = _code(x.dtype, "x")
    W, N, K2 = _matrix(qw, sw, _block(w_block), "qw")
    if K != K2:
        raise ValueError("inner dimensions differ")
    y, ldy, ycode = _output(out, out_dtype or x.dtype, M, N, x, stream)
    if stream is not None:
        _keep(stream, x, qw, sw, out)
    need = _u64()
    rc = _L.swz_linear_fp8_workspace_size(M, N, K, need)
    if rc == 0:
        need = need.value
        ws = _empty(need, torch.uint8, x, stream) if need else None
        rc = _L.swz_linear_fp8(x.data_ptr(), code, ldx, W, y.data_ptr(), ldy, ycode, M, N, K,
                               ws.data_ptr() if need else None, need, _handle(stream, x))
    if rc:
        raise _swz.SwzError(rc, "swz_linear_fp8")
    return _result("linear_fp8", y, out, x, qw, sw)


def linear_fp8_forward(x, w, *, out_dtype=None, stream=None):
    """(y, saved) of a layer in training: y = x W^T with x (M x K) quantised in
    row blocks and w (N x K) in square ones; ``saved`` holds x^T and W^T in 8
    bits for linear_fp8_backward."""
    if torch is None:
        _init()
    _here(x, w)
    qx, sx, qxt, sxt, M, K = _quantize(x, SWZ_BLOCK_ROW, "e4m3", True, stream)
    qw, sw, qwt, swt, N, K2 = _quantize(w, SWZ_BLOCK_SQUARE, "e4m3", True, stream)
    if K != K2:
        raise ValueError("inner dimensions differ")
    y = _product(_own(qx, sx, SWZ_E4M3, SWZ_BLOCK_ROW), _own(qw, sw, SWZ_E4M3, SWZ_BLOCK_SQUARE),
                 M, N, K, out_dtype or x.dtype, x, stream)
    return y, (qxt if qxt.shape[1] == M else qxt.narrow(1, 0, M), sxt,
               qwt if qwt.shape[1] == N else qwt.narrow(1, 0, N), swt)


def linear_fp8_backward(dy, saved, *, need_dx=True, need_dw=True, dx_dtype=None, dw_dtype=None,
                        stream=None):
    """(dx, dw) of linear_fp8_forward: dx = dy W (M x K; default dy's type)
    and dw = dy^T x (N x K; default fp32), dy quantised in row blocks along N
    and along the rows; None in place of one that is not needed."""
    qxt, sxt, qwt, swt = saved
    if torch is None:
        _init()
    _here(dy, *saved)
    M, N, _ = _rows(dy, "dy")
    if M != qxt.shape[1] or N != qwt.shape[1]:
        raise ValueError("dy does not have the shape of the layer's output")
    if stream is not None:
        _keep(stream, *saved)
    dx = dw = None
    if need_dx or need_dw:
        q, s, qt, st, _, _ = _quantize(dy, SWZ_BLOCK_ROW, "e4m3", need_dw, stream)
        if need_dx:
            W, K, _ = _matrix(qwt, swt, SWZ_BLOCK_SQUARE, "saved")
            dx = _product(_own(q, s, SWZ_E4M3, SWZ_BLOCK_ROW), W, M, K, N, dx_dtype or dy.dtype,
                          dy, stream)
        if need_dw:
            X, K, _ = _matrix(qxt, sxt, SWZ_BLOCK_ROW, "saved")
            dw = _product(_own(qt, st, SWZ_E4M3, SWZ_BLOCK_ROW), X, N, K, M,
                          dw_dtype or torch.float32, dy, stream)
    return dx, dw


def _with_rows(t):
    """t, or a copy of it whose rows are contiguous and apart."""
    return t if t.stride(1) == 1 and t.stride(0) >= t.shape[1] else t.contiguous()


_function = None


def fp8_linear(x, w):
    """y = x W^T with its gradient, for torch.autograd: x (..., K) and w (N, K),
    of any layout (copied where rows are not contiguous); forward and backward
    as linear_fp8_forward / linear_fp8_backward, the gradient of w in fp32
    rounded to w's type.  A second derivative raises."""
    global _function
    if _function is None:
        if torch is None:
            _init()

        class Fp8Linear(torch.autograd.Function):
            @staticmethod
            def forward(ctx, x, w):
                y, saved = linear_fp8_forward(_with_rows(x), _with_rows(w))
                ctx.save_for_backward(*saved)
                ctx.w_dtype = w.dtype
                return y

            @staticmethod
            @torch.autograd.function.once_differentiable
            def backward(ctx, dy):
                return linear_fp8_backward(
                    _with_rows(dy), ctx.saved_tensors, need_dx=ctx.needs_input_grad[0],
                    need_dw=ctx.needs_input_grad[1], dw_dtype=ctx.w_dtype)

        _function = Fp8Linear
    flat = x.reshape(math.prod(x.shape[:-1]), x.shape[-1])
    return _function.apply(flat, w).reshape(*x.shape[:-1], w.shape[0])


def newton_schulz(G, steps=5, coefficients=(3.4445, -4.7750, 2.0315), eps=1e-7, *, out=None,
                  out_dtype=None, tile=0, debug_flags=0, timeout_ms=0, stream=None):
    """The orthogonalised update of G (m x n, or a stack batch x m x n; fp16,
    bf16 or fp32, contiguous rows): X = G / (|G|_F + eps), then ``steps`` times
    X = a X + (b A + c A^2) X with A = X X^T (on the right with X^T X when m >
    n), ``coefficients`` = (a, b, c).  ``out`` (G's shape; may lie over G in any
    way) or ``out_dtype`` (default bf16).

    The products take fp16 operands with fp32 sums, whatever the types of G and
    the result: after five steps X is 0.06 to 0.15 % off, next to the 0.17 % that a
    bf16 result's rounding costs."""
    if torch is None:
        _init()
    if G.dim() not in (2, 3):
        raise ValueError("G: 2-D or 3-D tensor expected")
    _here(G, out)
    if stream is not None:
        _keep(stream, G, out)
    if max(G.shape) > INT_MAX:
        raise ValueError("G: more than 2^31 - 1 matrices, rows or columns")
    _in_range(debug_flags, timeout_ms, steps, tile)
    code = _code(G.dtype, "G")
    fresh = out is None
    if fresh:
        ycode = _code(out_dtype or torch.bfloat16, "out_dtype")
        out = _empty(G.shape, out_dtype or torch.bfloat16, G, stream)
    else:
        ycode = _code(out.dtype, "out")
        if out.shape != G.shape:
            raise ValueError(f"out: shape {tuple(G.shape)} expected")
    g, y = (t if t.dim() == 3 else t.unsqueeze(0) for t in (G, out))
    batch, m, n = g.shape
    ld = []
    for t, what in ((g, "G"), (y, "out")):
        sb, sm, sn = t.stride()
        if (n > 1 and sn != 1) or (m > 1 and sm < n) or (batch > 1 and sb < (m - 1) * sm + n):
            raise ValueError(f"{what}: contiguous rows that do not overlap expected")
        ld.append((sm if m > 1 else max(n, 1), sb if batch > 1 else 0))
    a, b, c = coefficients
    rc, need = swz_newton_schulz_workspace_size(batch, m, n)
    _swz._check(rc, "swz_newton_schulz_workspace_size")
    ws = _empty((max(need, 1),), torch.uint8, G, stream)
    opts = swz_newton_schulz_opts(tile, debug_flags, timeout_ms)
    _swz._check(_L.swz_newton_schulz(g.data_ptr(), code, *ld[0], y.data_ptr(), ycode, *ld[1], batch, m,
                                     n, steps, a, b, c, eps, opts, ws.data_ptr(), need,
                                     _handle(stream, G)), "swz_newton_schulz")
    return _result("newton_schulz", out, None if fresh else out, G)

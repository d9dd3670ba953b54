"""Linear layers in 8-bit integers on torch tensors: quantisation by rows (the
tokens of activations, the output channels of weights) and the product with a
scale for each row of either operand, over the C entry points of include/swz.h
(argument marshalling only; every computation runs in the library's kernels).

Matrices are ``torch.int8`` tensors of shape (rows, K) whose rows start on
multiples of 16 bytes (``quantize_int8`` makes them so; ``int8_empty`` allocates
one), their scales fp32 tensors of shape (rows,).  All operands of a call are on
the current device; ``stream`` is as in ``linear``.  The operators have no
gradient: a backward through what they return raises (``out`` takes values only),
through the product of rows that were quantised from x as well; weights that are kept
for serving are quantised from a detached tensor or under ``torch.no_grad``.
"""
from __future__ import annotations

import ctypes

import thread_block_smem_gb300 as _swz

from . import linear as _lin

MAX_K = 131071  # longest sum that fits 32 bits


class swz_gemm_int8_opts(ctypes.Structure):
    _fields_ = [("order", ctypes.c_int), ("group", ctypes.c_int), ("tile", ctypes.c_int),
                ("split_k", ctypes.c_int), ("debug_flags", ctypes.c_uint32),
                ("timeout_ms", ctypes.c_uint32)]


def declare(L):
    """Argument types of this module's entry points on the loaded library."""
    i, i64, u64, vp = ctypes.c_int, ctypes.c_int64, ctypes.c_uint64, ctypes.c_void_p
    L.swz_quantize_int8.argtypes = [vp, i, i64, i, i, vp, i64, vp, vp]
    L.swz_gemm_int8.argtypes = [vp, i64, vp, vp, i64, vp, vp, i64, i, i, i, i,
                                ctypes.POINTER(swz_gemm_int8_opts), vp, u64, vp]
    L.swz_gemm_int8_workspace_size.argtypes = [i, i, i, i, ctypes.POINTER(u64)]
    L.swz_gemm_int8_workspace_size_ex.argtypes = [i, i, i, ctypes.POINTER(swz_gemm_int8_opts),
                                                  ctypes.POINTER(u64)]
    L.swz_linear_int8.argtypes = [vp, i, i64, vp, i64, vp, vp, i64, i, i, i, i, vp, u64, vp]
    L.swz_linear_int8_workspace_size.argtypes = [i, i, i, ctypes.POINTER(u64)]


# ---- raw mirrors ----------------------------------------------------------------
def swz_quantize_int8(x, dtype, ldx, M, K, q, ldq, scales, stream=0):
    if not _lin._ints(dtype, M, K):
        return _swz.SWZ_EINVAL
    return _swz.lib().swz_quantize_int8(x, dtype, ldx, M, K, q, ldq, scales, stream)


def swz_gemm_int8(A, lda, sa, B, ldb, sb, C, ldc, c_dtype, M, N, K, opts, workspace,
                  workspace_bytes, stream=0):
    if not _lin._ints(c_dtype, M, N, K):
        return _swz.SWZ_EINVAL
    return _swz.lib().swz_gemm_int8(A, lda, sa, B, ldb, sb, C, ldc, c_dtype, M, N, K,
                                    ctypes.byref(opts) if opts is not None else None, workspace,
                                    workspace_bytes, stream)


def swz_linear_int8(x, dtype, ldx, W, ldw, sw, y, ldy, y_dtype, M, N, K, workspace,
                    workspace_bytes, stream=0):
    if not _lin._ints(dtype, y_dtype, M, N, K):
        return _swz.SWZ_EINVAL
    return _swz.lib().swz_linear_int8(x, dtype, ldx, W, ldw, sw, y, ldy, y_dtype, M, N, K,
                                      workspace, workspace_bytes, stream)


def _size(fn, *sizes):
    if not _lin._ints(*sizes):
        return _swz.SWZ_EINVAL, 0
    b = ctypes.c_uint64(0)
    rc = fn(*sizes, ctypes.byref(b))
    return rc, b.value


def swz_gemm_int8_workspace_size(M, N, K, tile=0):
    return _size(_swz.lib().swz_gemm_int8_workspace_size, M, N, K, tile)


def swz_gemm_int8_workspace_size_ex(M, N, K, opts=None):
    if not _lin._ints(M, N, K):
        return _swz.SWZ_EINVAL, 0
    b = ctypes.c_uint64(0)
    rc = _swz.lib().swz_gemm_int8_workspace_size_ex(
        M, N, K, ctypes.byref(opts) if opts is not None else None, ctypes.byref(b))
    return rc, b.value


def swz_linear_int8_workspace_size(M, N, K):
    return _size(_swz.lib().swz_linear_int8_workspace_size, M, N, K)


# ---- operators --------------------------------------------------------------------
def int8_empty(rows, cols, device="cuda"):
    """Uninitialised int8 (rows, cols) tensor whose rows start on multiples of 16 bytes."""
    if _lin.torch is None:
        _lin._init()
    return _lin.fp8_empty(rows, cols, _lin.torch.int8, device)


def _matrix(q, scales, what):
    """(address, bytes from row to row, address of the scales, rows, columns), checked."""
    torch = _lin.torch
    if q.dtype != torch.int8:
        raise TypeError(f"{what}: int8 expected")
    m, k, ld = _lin._rows(q, what)
    if m <= 1 or k == 0:  # no second row whose place matters
        ld = (k + 15) // 16 * 16
    at = q.data_ptr()
    if ld % 16 or at % 16:
        raise ValueError(f"{what}: rows must start on multiples of 16 bytes")
    if k > MAX_K:
        raise ValueError(f"{what}: more than {MAX_K} columns, whose products' sum may not fit 32 bits")
    if scales.dtype != torch.float32 or not scales.is_cuda:
        raise TypeError(f"{what}: fp32 CUDA scales expected")
    if scales.dim() != 1 or scales.shape[0] != m:
        raise ValueError(f"{what}: scales of shape {(m,)} expected, got {tuple(scales.shape)}")
    if m > 1 and scales.stride(0) != 1:
        raise ValueError(f"{what}: contiguous scales expected")
    return at, ld, scales.data_ptr(), m, k


def quantize_int8(x, *, stream=None):
    """(q, scales) of x (M x K; fp16, bf16 or fp32, contiguous rows), a scale for
    each row.  For a row with largest magnitude amax: ac = max(amax, 2^-96),
    r = 127 / ac, scale = ac / 127, q = x r rounded to the nearest whole number,
    ties to even.  A row with an infinity or NaN gets zeros and the scale NaN."""
    if _lin.torch is None:
        _lin._init()
    torch = _lin.torch
    _lin._here(x)
    M, K, ldx = _lin._rows(x, "x")
    code = _lin._code(x.dtype, "x")
    if stream is not None:
        _lin._keep(stream, x)
    ldq = (K + 15) // 16 * 16
    # (made with its strides: cutting the rows afterwards cost a call 7 us)
    with _lin._on(stream):
        q = torch.empty_strided((M, K), (ldq, 1), dtype=torch.int8, device=x.device)
        s = torch.empty(M, dtype=torch.float32, device=x.device)
    rc = _lin._L.swz_quantize_int8(x.data_ptr(), code, ldx, M, K, q.data_ptr(), ldq, s.data_ptr(),
                                   _lin._handle(stream, x))
    if rc:
        raise _swz.SwzError(rc, "swz_quantize_int8")
    return q, _lin._no_gradient("quantize_int8", s, x)


def gemm_int8(a, sa, b, sb, *, out=None, out_dtype=None, order="serpentine", group=8, tile=0,
              split_k=0, debug_flags=0, timeout_ms=0, stream=None):
    """C = A B^T (M x N) of 8-bit integers: a (M x K) with the scales sa of its
    rows, b (N x K) with the scales sb of its rows; the sums are exact (K up to
    131071).  ``out`` (M x N, contiguous rows) or ``out_dtype`` (fp32, bf16 or
    fp16; default bf16).  ``order``, ``group``: the order of the output tiles, as
    in ``gemm``; ``tile``, ``split_k``: see swz_gemm_int8_opts (0 = automatic)."""
    if _lin.torch is None:
        _lin._init()
    torch = _lin.torch
    _lin._here(a, sa, b, sb, out)
    pa, lda, psa, M, K = _matrix(a, sa, "a")
    pb, ldb, psb, N, K2 = _matrix(b, sb, "b")
    if K != K2:
        raise ValueError("inner dimensions differ")
    order = _swz._order(order)
    _lin._in_range(debug_flags, timeout_ms, order, group, tile, split_k)
    C, ldc, code = _lin._output(out, out_dtype or torch.bfloat16, M, N, a, stream)
    if stream is not None:
        _lin._keep(stream, a, sa, b, sb, out)
    opts = swz_gemm_int8_opts(order, group, tile, split_k, debug_flags, timeout_ms)
    need = _lin._u64()
    rc = _lin._L.swz_gemm_int8_workspace_size_ex(M, N, K, opts, need)
    if rc == 0:
        need = need.value
        ws = _lin._empty(need, torch.uint8, a, stream) if need else None
        rc = _lin._L.swz_gemm_int8(pa, lda, psa, pb, ldb, psb, C.data_ptr(), ldc, code, M, N, K, opts,
                                   ws.data_ptr() if need else None, need, _lin._handle(stream, a))
    if rc:
        raise _swz.SwzError(rc, "swz_gemm_int8")
    return _lin._result("gemm_int8", C, out, a, sa, b, sb)


def linear_int8(x, qw, sw, *, out=None, out_dtype=None, stream=None):
    """y = x W^T (M x N): x (M x K; fp16, bf16 or fp32) is quantised by rows as in
    ``quantize_int8`` and multiplied by W (N x K) kept as (qw, sw).  ``out`` (may lie
    over x in any way; over qw or sw it is refused) or ``out_dtype`` (default: x's
    type)."""
    if _lin.torch is None:
        _lin._init()
    _lin._here(x, qw, sw, out)
    M, K, ldx = _lin._rows(x, "x")
    code = _lin._code(x.dtype, "x")
    pw, ldw, psw, N, K2 = _matrix(qw, sw, "qw")
    if K != K2:
        raise ValueError("inner dimensions differ")
    y, ldy, ycode = _lin._output(out, out_dtype or x.dtype, M, N, x, stream)
    if stream is not None:
        _lin._keep(stream, x, qw, sw, out)
    need = _lin._u64()
    rc = _lin._L.swz_linear_int8_workspace_size(M, N, K, need)
    if rc == 0:
        need = need.value
        ws = _lin._empty(need, _lin.torch.uint8, x, stream) if need else None
        call = (x.data_ptr(), code, ldx, pw, ldw, psw, y.data_ptr(), ldy, ycode, M, N, K)
        rc = _lin._L.swz_linear_int8(*call, ws.data_ptr() if need else None, need,
                                     _lin._handle(stream, x))
        if rc == _swz.SWZ_EINVAL and need == 0 and out is not None:
            # out lies over x, which is then quantised before out is written
            need = 256 + M * ((K + 15) // 16 * 16)
            ws = _lin._empty(need, _lin.torch.uint8, x, stream)
            rc = _lin._L.swz_linear_int8(*call, ws.data_ptr(), need, _lin._handle(stream, x))
    if rc:
        raise _swz.SwzError(rc, "swz_linear_int8")
    return _lin._result("linear_int8", y, out, x, qw, sw)

"""Products of 8-bit floating point matrices with a scale for each block of 128 (the C ABI of include/fp8.h).

Argument marshalling only, as in :mod:`dense_fp32_matrix_major_gb300.experts`, whose conventions on streams, devices,
gradients and errors this module shares. A linear layer's step, y = x W^T, from weights that were quantised once::

    w8 = fp8.quantize(w, "blocks")                           # out x in, scales per 128 x 128
    y = fp8.gemm(fp8.quantize(x, "rows"), w8, transB=True)

and its gradients::

    dx = fp8.gemm(fp8.quantize(dy, "rows", dtype=torch.float8_e5m2), w8)
    dw = fp8.gemm_wgrad(fp8.quantize(dy, "columns", dtype=torch.float8_e5m2), fp8.quantize(x, "columns"))

With ``offsets`` (of :func:`dense_fp32_matrix_major_gb300.experts.sort`) the same calls make one product per expert.
"""

from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from .experts import TYPES, _check, _contiguous, _empty, _stream_handle
from .sgemm import lib

SGEMM_FP8_E4M3 = 0
SGEMM_FP8_E5M2 = 1
SGEMM_FP8_ROWS = 0
SGEMM_FP8_COLUMNS = 1
SGEMM_FP8_BLOCKS = 2
SGEMM_FP8_BLOCK_SIZE = 128

FP8_TYPES = {torch.float8_e4m3fn: SGEMM_FP8_E4M3, torch.float8_e5m2: SGEMM_FP8_E5M2}
BLOCK_SHAPES = {"rows": SGEMM_FP8_ROWS, "columns": SGEMM_FP8_COLUMNS, "blocks": SGEMM_FP8_BLOCKS}

# Every function that include/fp8.h declares, with its ctypes signature.
_i64, _int, _vp = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p
SIGNATURES = {
    "sgemm_fp8_quantize": (_int, [_int, _int, _int, _int, _i64, _i64, _i64, _vp, _i64, _i64, _i64, _vp, _vp, _i64,
                                  _i64, _vp, _vp]),
    "sgemm_fp8_blocks": (_i64, [_i64, _i64]),
    "sgemm_fp8_gemm": (_int, [_int, _int, _int, _int, _i64, _i64, _i64, _i64, _vp, _vp, _i64, _vp, _vp, _i64, _i64,
                              _vp, _vp, _i64, _vp]),
    "sgemm_fp8_gemm_wgrad": (_int, [_int, _int, _int, _i64, _i64, _i64, _i64, _vp, _vp, _i64, _vp, _vp, _i64, _vp,
                                    _vp, _i64, _i64, _vp]),
}
for _name, (_res, _args) in SIGNATURES.items():
    _fn = getattr(lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args

_FP32 = (torch.float32,)
_INT32 = (torch.int32,)


class Quantized(NamedTuple):
    """A matrix (or stack of matrices) in 8-bit floating point (see :func:`quantize`)."""

    values: torch.Tensor  # float8_e4m3fn or float8_e5m2
    scales: torch.Tensor  # float32: blocks x rows, blocks x columns, or blocks of rows x blocks of columns


def _blocks(n):
    return (n + 127) // 128


def _pitch(cols):
    """Row stride of a matrix of these sizes whose own says nothing (one row, no elements)."""
    return max(-(-cols // 16) * 16, 16)


def _strides(t, name, dtypes, dims):
    """Row and item stride of a 2-D or 3-D CUDA tensor of row-major matrices."""
    if not isinstance(t, torch.Tensor) or t.dtype not in dtypes or t.dim() not in dims or not t.is_cuda:
        raise TypeError(f"{name} must be a {' or '.join(f'{d}-D' for d in dims)} CUDA tensor of "
                        f"{' or '.join(str(d) for d in dtypes)}")
    strides = t.stride()
    rows, cols = t.shape[-2:]
    if cols > 1 and strides[-1] != 1:
        raise ValueError(f"{name} must have unit column stride (row-major)")
    if rows == 0 or cols == 0:
        return _pitch(cols), 0
    return (strides[-2] if rows > 1 else _pitch(cols)), (strides[0] if len(strides) == 3 else 0)


def _operand(t, name, dims, block):
    """(type, row stride, item stride, values pointer, scales pointer) of a product's operand."""
    if not isinstance(t, Quantized):
        raise TypeError(f"{name} must be a fp8.Quantized")
    values, scales = t
    ld, stride = _strides(values, name, FP8_TYPES, dims)
    shape = values.shape
    ptr = values.data_ptr()
    if ld % 16 or ptr % 16 or (stride % 16 and shape[0] > 1):
        raise ValueError(f"{name}'s rows must start on 16-byte boundaries (as fp8.quantize lays them out)")
    if block == "rows":
        want = (_blocks(shape[1]), shape[0])
    elif block == "columns":
        want = (_blocks(shape[0]), shape[1])
    else:
        want = (*shape[:-2], _blocks(shape[-2]), _blocks(shape[-1]))
    return FP8_TYPES[values.dtype], ld, stride, ptr, _contiguous(scales, f"{name}'s scales", _FP32, want)


def _out(out, shape, dtype, like, stream):
    """(tensor, row stride, item stride) of a product's result, ``out`` or a new tensor."""
    rows, cols = shape[-2:]
    if out is None:
        if dtype not in TYPES:
            raise TypeError("dtype must be float32, bfloat16 or float16")
        return (_empty(shape, dtype, like.device, stream), cols if rows > 1 and cols else _pitch(cols),
                rows * cols if len(shape) == 3 else 0)
    if not isinstance(out, torch.Tensor) or out.dtype not in TYPES:
        raise TypeError("out must be a float32, bfloat16 or float16 tensor")
    if tuple(out.shape) != shape:
        raise ValueError("out has the wrong shape")
    return (out, *_strides(out, "out", TYPES, (len(shape),)))


def quantize(x, block="rows", *, dtype=torch.float8_e4m3fn, pow2=False, offsets=None, out=None, stream=None):
    """``x`` in 8-bit floating point with one fp32 scale per block of 128; returns a :class:`Quantized`.

    ``block`` is "rows" (1 x 128; scales ceil(cols / 128) x rows), "columns" (128 x 1; scales ceil(rows / 128) x
    cols) or "blocks" (128 x 128; scales ceil(rows / 128) x ceil(cols / 128)), ``x`` a float32, bfloat16 or float16
    matrix, or a stack of them with "blocks". The scale is the block's largest finite magnitude over the type's
    largest value, with ``pow2`` the power of two not below that; infinities and NaN become NaN. With ``offsets``
    (int32, experts + 1 long, rows sorted by expert) and "columns" every group starts a block of its own, stored as
    128 rows with zeros at the end: the layout :func:`gemm_wgrad` reads. New values have rows that start 16 bytes
    apart, as the products want them.
    """
    if block not in BLOCK_SHAPES:
        raise ValueError("block must be rows, columns or blocks")
    if dtype not in FP8_TYPES:
        raise TypeError("dtype must be torch.float8_e4m3fn or torch.float8_e5m2")
    ldx, stride_x = _strides(x, "x", TYPES, (2, 3) if block == "blocks" else (2,))
    rows, cols = x.shape[-2:]
    if rows == 1:
        ldx = max(cols, 1)
    items = x.shape[0] if x.dim() == 3 else 1
    experts, off = 1, 0
    stored = rows
    if offsets is not None:
        if block != "columns":
            raise ValueError('offsets go with block="columns"')
        off = _contiguous(offsets, "offsets", _INT32)
        if offsets.dim() != 1 or offsets.shape[0] < 2:
            raise ValueError("offsets must be experts + 1 long")
        experts = offsets.shape[0] - 1
        stored = 128 * lib.sgemm_fp8_blocks(rows, experts)
    lead = x.shape[:-2]
    pow2 = 1 if pow2 else 0
    shape = (_blocks(cols), rows) if block == "rows" else \
        (_blocks(stored), cols) if block == "columns" else (*lead, _blocks(rows), _blocks(cols))
    if out is None:
        ldq = max(-(-cols // 16) * 16, 16)
        values = _empty((*lead, stored, ldq), dtype, x.device, stream)
        scales = _empty(shape, torch.float32, x.device, stream)
        out = Quantized(values if ldq == cols else values[..., :cols], scales)
        stride_q, sp = (stored * ldq if lead else 0), scales.data_ptr()
    else:
        if not isinstance(out, Quantized) or out.values.dtype != dtype:
            raise TypeError(f"out must be a fp8.Quantized of {dtype}")
        values, scales = out
        if tuple(values.shape) != (*lead, stored, cols):
            raise ValueError("out has the wrong shape")
        ldq, stride_q = _strides(values, "out", FP8_TYPES, (x.dim(),))
        sp = _contiguous(scales, "out's scales", _FP32, shape)
    _check(lib.sgemm_fp8_quantize(TYPES[x.dtype], BLOCK_SHAPES[block], FP8_TYPES[dtype], pow2, items, rows, cols,
                                  x.data_ptr(), ldx, stride_x, experts, off, values.data_ptr(), ldq, stride_q, sp,
                                  _stream_handle(stream, x, offsets, values, scales)),
           "sgemm_fp8_quantize")
    return out


def gemm(a, b, offsets=None, out=None, *, transB=False, dtype=torch.bfloat16, stream=None):
    """out = a @ op(b), or with ``offsets`` one product per expert: out[s] = a[s] @ op(b[e]), zero outside groups.

    ``a`` holds rows x K quantised in "rows", ``b`` K x N (N x K when ``transB``), or experts of them, quantised in
    "blocks". The result is of ``dtype`` (float32, bfloat16 or float16), or ``out``'s. The gradient of ``a`` is the
    same call on the output's gradient with ``transB`` the other way round.
    """
    ta, lda, _, ap, sa = _operand(a, "a", (2,), "rows")
    tb, ldb, stride, bp, sb = _operand(b, "b", (2,) if offsets is None else (3,), "blocks")
    rows, K = a.values.shape
    shape = b.values.shape
    N, K2 = shape[-2:] if transB else shape[:-3:-1]
    if K != K2:
        raise ValueError(f"inner dimensions differ: {K} vs {K2}")
    E, off = 1, 0
    if offsets is not None:
        E = shape[0]
        off = _contiguous(offsets, "offsets", _INT32, (E + 1,))
    out, ldc, _ = _out(out, (rows, N), dtype, a.values, stream)
    _check(lib.sgemm_fp8_gemm(TYPES[out.dtype], 1 if transB else 0, ta, tb, rows, N, K, E, off, ap, lda, sa, bp, ldb,
                              stride, sb, out.data_ptr(), ldc, _stream_handle(stream, *a, *b, offsets, out)),
           "sgemm_fp8_gemm")
    return out


def gemm_wgrad(a, b, offsets=None, out=None, *, dtype=torch.float32, stream=None):
    """out = a^T @ b, or with ``offsets`` out[e] = a_e^T @ b_e over the rows of each group (zeros for empty ones).

    ``a`` holds rows x M and ``b`` rows x N, both quantised in "columns", with the same ``offsets``. The gradient of
    :func:`gemm`'s b is ``gemm_wgrad(a, dout)``, or ``gemm_wgrad(dout, a)`` for ``transB``. The result is of
    ``dtype``, or ``out``'s.
    """
    ta, lda, _, ap, sa = _operand(a, "a", (2,), "columns")
    tb, ldb, _, bp, sb = _operand(b, "b", (2,), "columns")
    rows, M = a.values.shape
    if b.values.shape[0] != rows:
        raise ValueError(f"a has {rows} rows, b {b.values.shape[0]}")
    N = b.values.shape[1]
    E, off = 1, 0
    if offsets is not None:
        off = _contiguous(offsets, "offsets", _INT32)
        if offsets.dim() != 1 or offsets.shape[0] < 2:
            raise ValueError("offsets must be experts + 1 long")
        if rows % 128:
            raise ValueError("operands with offsets hold whole blocks of 128 rows (as fp8.quantize lays them out)")
        E = offsets.shape[0] - 1
    out, ldc, stride = _out(out, (M, N) if offsets is None else (E, M, N), dtype, a.values, stream)
    _check(lib.sgemm_fp8_gemm_wgrad(TYPES[out.dtype], ta, tb, rows, M, N, E, off, ap, lda, sa, bp, ldb, sb,
                                    out.data_ptr(), ldc, stride, _stream_handle(stream, *a, *b, offsets, out)),
           "sgemm_fp8_gemm_wgrad")
    return out

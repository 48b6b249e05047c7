"""Operators of a mixture-of-experts layer on torch CUDA tensors (the C ABI of include/experts.h).

Argument marshalling only, as in :mod:`dense_fp32_matrix_major_gb300.sgemm`, whose library, errors and stream
convention this module shares: calls are enqueued on ``stream`` (the current stream by default), outputs that
are not given are allocated by PyTorch on that stream, there is no CPU fallback.

A layer's forward pass::

    r = experts.sort(ids, num_experts)             # ids: tokens x top_k
    xs = experts.gather(x, r)                      # rows in expert order
    h = experts.gemm(xs, w1, r.offsets)            # one product per expert
    ...                                            # activation
    y = experts.combine(experts.gemm(h, w2, r.offsets), weights, r)

and its gradients: :func:`combine_grad`, :func:`gemm` with ``transB`` the other way round for the rows,
:func:`gemm_wgrad` for the experts' matrices, :func:`gather_grad`. :func:`w4_matvec` serves single tokens from
4-bit matrices. The calls record no gradients of their own: in a model they stand inside a torch.autograd.Function
(an input that requires a gradient elsewhere draws a warning).
"""

from __future__ import annotations

import ctypes
import warnings
from typing import NamedTuple

import torch

from .sgemm import SgemmError, lib

SGEMM_TYPE_F32 = 0
SGEMM_TYPE_BF16 = 1
SGEMM_TYPE_F16 = 2
SGEMM_EXPERTS_MAX = 4096
SGEMM_TOP_K_MAX = 64
SGEMM_W4_ROWS_MAX = 65535

TYPES = {torch.float32: SGEMM_TYPE_F32, torch.bfloat16: SGEMM_TYPE_BF16, torch.float16: SGEMM_TYPE_F16}

# Every function that include/experts.h declares, with its ctypes signature.
_i64, _int, _vp, _sz = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t
SIGNATURES = {
    "sgemm_experts_sort": (_int, [_vp, _int, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _sz, _vp]),
    "sgemm_experts_sort_workspace": (_sz, [_i64, _i64]),
    "sgemm_experts_gather": (_int, [_int, _i64, _i64, _i64, _i64, _vp, _i64, _vp, _vp, _vp, _i64, _vp]),
    "sgemm_experts_combine": (_int, [_int, _i64, _i64, _i64, _i64, _vp, _i64, _vp, _vp, _vp, _vp, _i64, _vp]),
    "sgemm_experts_combine_grad": (_int, [_int, _i64, _i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _vp,
                                          _i64, _vp, _vp]),
    "sgemm_experts_gemm": (_int, [_int, _int, _i64, _i64, _i64, _i64, _vp, _vp, _i64, _vp, _i64, _i64, _vp, _i64,
                                  _vp]),
    "sgemm_experts_gemm_wgrad": (_int, [_int, _i64, _i64, _i64, _i64, _vp, _vp, _i64, _vp, _i64, _vp, _i64, _i64,
                                        _vp]),
    "sgemm_w4_matvec": (_int, [_int, _i64, _i64, _i64, _i64, _i64, _vp, _vp, _i64, _vp, _vp, _int, _vp, _vp, _i64,
                               _vp]),
}
for _name, (_res, _args) in SIGNATURES.items():
    _fn = getattr(lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args


class Routing(NamedTuple):
    """Pairs sorted by expert (see :func:`sort`)."""

    offsets: torch.Tensor  # experts + 1, int32: group e holds slots offsets[e] .. offsets[e + 1] - 1
    order: torch.Tensor    # tokens * top_k, int32: the pair (token * top_k + choice) at each slot
    slot: torch.Tensor     # tokens x top_k, int32: the slot of each pair


# The current stream's handle without a Stream object (which costs 3 us).
_current_stream = torch._C._cuda_getCurrentRawStream


def _stream_handle(stream, *tensors):
    """The stream's handle; every tensor (or None) must be on the current device, which the library launches on.

    Warns where PyTorch would expect a gradient to flow through the call."""
    device = torch.cuda.current_device()
    lost = False
    for t in tensors:
        if t is not None:
            if t.get_device() != device:
                raise ValueError(f"tensors are on cuda:{t.get_device()}, the current device is cuda:{device}")
            lost |= t.requires_grad
    if lost and torch.is_grad_enabled():
        warnings.warn("an input requires a gradient, but these calls record none: the result is cut from the graph "
                      "(call them inside torch.autograd.Function or torch.no_grad())", stacklevel=3)
    if stream is None:
        return _current_stream(device)
    if stream.device_index != device:
        raise ValueError(f"the stream is on cuda:{stream.device_index}, the current device is cuda:{device}")
    return stream.cuda_stream


def _check(rc, what):
    if rc:
        raise SgemmError(rc, what)


def _empty(shape, dtype, device, stream):
    """A new tensor that belongs to the stream its first use is enqueued on."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _rows(t, name, dtype=None):
    """Type code and row stride of a 2-D tensor with unit column stride."""
    if not isinstance(t, torch.Tensor) or t.dtype not in TYPES or t.dim() != 2:
        raise TypeError(f"{name} must be a 2-D float32, bfloat16 or float16 tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}")
    if not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    rows, cols = t.shape
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have unit column stride (row-major)")
    return TYPES[t.dtype], t.stride(0) if rows > 1 else max(cols, 1)


def _matrices(t, name, dtype):
    """Row and item stride of a 3-D tensor of row-major matrices."""
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.dim() != 3 or not t.is_cuda:
        raise TypeError(f"{name} must be a 3-D {dtype} CUDA tensor")
    items, rows, cols = t.shape
    if cols > 1 and t.stride(2) != 1:
        raise ValueError(f"{name} must have unit column stride")
    return (t.stride(1) if rows > 1 else max(cols, 1)), (t.stride(0) if items > 1 else 0)


def _contiguous(t, name, dtypes, shape=None):
    if not isinstance(t, torch.Tensor) or t.dtype not in dtypes or not t.is_cuda or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous CUDA tensor of {' or '.join(str(d) for d in dtypes)}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}")
    return t.data_ptr()


_INT32 = (torch.int32,)


def _routing(r):
    """(tokens, top_k, experts, slot pointer, offsets pointer) of a Routing."""
    slot = _contiguous(r.slot, "routing.slot", _INT32)
    offsets = _contiguous(r.offsets, "routing.offsets", _INT32)
    if r.slot.dim() != 2 or r.offsets.dim() != 1 or r.offsets.shape[0] < 2:
        raise ValueError("routing.slot must be tokens x top_k, routing.offsets experts + 1 long")
    return r.slot.shape[0], r.slot.shape[1], r.offsets.shape[0] - 1, slot, offsets


def sort(ids, experts, stream=None):
    """Sort (token, choice) pairs by expert, stably; returns a :class:`Routing`.

    ``ids`` is a contiguous tokens x top_k int32 or int64 CUDA tensor. A choice whose id is not in 0 ..
    experts - 1 is dropped: it is sorted last and takes part in nothing.
    """
    ptr = _contiguous(ids, "ids", (torch.int32, torch.int64))
    if ids.dim() != 2:
        raise ValueError("ids must be tokens x top_k")
    tokens, top_k = ids.shape
    pairs = tokens * top_k
    experts = int(experts)
    if experts < 1:
        raise ValueError("experts must be at least 1")
    device = ids.device
    offsets = _empty((experts + 1,), torch.int32, device, stream)
    order = _empty((pairs,), torch.int32, device, stream)
    slot = _empty((tokens, top_k), torch.int32, device, stream)
    need = lib.sgemm_experts_sort_workspace(pairs, experts)
    space = _empty((need // 4,), torch.int32, device, stream) if need else None
    _check(lib.sgemm_experts_sort(ptr, 64 if ids.dtype == torch.int64 else 32, tokens, top_k, experts,
                                  offsets.data_ptr(), order.data_ptr(), slot.data_ptr(),
                                  space.data_ptr() if need else 0, need, _stream_handle(stream, ids)),
           "sgemm_experts_sort")
    return Routing(offsets, order, slot)


def gather(x, routing, out=None, stream=None):
    """Rows of ``x`` (tokens x width) in slot order: tokens * top_k x width, zero for dropped pairs."""
    code, ldx = _rows(x, "x")
    tokens, top_k, experts, slot, offsets = _routing(routing)
    width = x.shape[1]
    if x.shape[0] != tokens:
        raise ValueError(f"x has {x.shape[0]} rows for {tokens} tokens")
    if out is None:
        out = _empty((tokens * top_k, width), x.dtype, x.device, stream)
    _, ldo = _rows(out, "out", x.dtype)
    if tuple(out.shape) != (tokens * top_k, width):
        raise ValueError("out has the wrong shape")
    _check(lib.sgemm_experts_gather(code, tokens, top_k, experts, width, x.data_ptr(), ldx, slot, offsets,
                                    out.data_ptr(), ldo, _stream_handle(stream, x, out, routing.slot, routing.offsets)),
           "sgemm_experts_gather")
    return out


def _combine(h, weights, routing, out, stream):
    code, ldh = _rows(h, "h")
    tokens, top_k, experts, slot, offsets = _routing(routing)
    width = h.shape[1]
    if h.shape[0] != tokens * top_k:
        raise ValueError(f"h has {h.shape[0]} rows for {tokens * top_k} pairs")
    w = 0
    if weights is not None:
        w = _contiguous(weights, "weights", (torch.float32,), (tokens, top_k))
    if out is None:
        out = _empty((tokens, width), h.dtype, h.device, stream)
    _, ldo = _rows(out, "out", h.dtype)
    if tuple(out.shape) != (tokens, width):
        raise ValueError("out has the wrong shape")
    _check(lib.sgemm_experts_combine(code, tokens, top_k, experts, width, h.data_ptr(), ldh, w, slot, offsets,
                                     out.data_ptr(), ldo,
                                     _stream_handle(stream, h, weights, out, routing.slot, routing.offsets)),
           "sgemm_experts_combine")
    return out


def gather_grad(dxs, routing, out=None, stream=None):
    """Gradient of :func:`gather`'s x: each token's rows of ``dxs`` summed (dropped pairs left out)."""
    return _combine(dxs, None, routing, out, stream)


def combine(h, weights, routing, out=None, stream=None):
    """y[t] = sum over choices j of weights[t, j] * h[slot[t, j]], dropped pairs left out.

    ``h`` is tokens * top_k x width in slot order, ``weights`` a contiguous tokens x top_k float32 tensor.
    """
    if weights is None:
        raise TypeError("weights must be a contiguous CUDA tensor of torch.float32")
    return _combine(h, weights, routing, out, stream)


def combine_grad(dy, h, weights, routing, stream=None):
    """Gradients of :func:`combine`: (dh of h's shape and type, dweights tokens x top_k float32)."""
    code, lddy = _rows(dy, "dy")
    _, ldh = _rows(h, "h", dy.dtype)
    tokens, top_k, experts, slot, offsets = _routing(routing)
    width = h.shape[1]
    if h.shape[0] != tokens * top_k or tuple(dy.shape) != (tokens, width):
        raise ValueError("dy must be tokens x width and h tokens * top_k x width")
    w = _contiguous(weights, "weights", (torch.float32,), (tokens, top_k))
    dh = _empty(tuple(h.shape), h.dtype, h.device, stream)
    dw = _empty((tokens, top_k), torch.float32, h.device, stream)
    _check(lib.sgemm_experts_combine_grad(code, tokens, top_k, experts, width, dy.data_ptr(), lddy, h.data_ptr(), ldh,
                                          w, slot, offsets, dh.data_ptr(), max(width, 1), dw.data_ptr(),
                                          _stream_handle(stream, dy, h, weights, routing.slot, routing.offsets)),
           "sgemm_experts_combine_grad")
    return dh, dw


def gemm(a, b, offsets, out=None, *, transB=False, stream=None):
    """One product per group: out[s] = a[s] @ op(b[e]) for offsets[e] <= s < offsets[e + 1], zero elsewhere.

    ``a`` is rows x K, ``b`` experts x K x N (experts x N x K when ``transB``), ``offsets`` int32, experts + 1
    long. The gradient of ``a`` is the same call on the output's gradient with ``transB`` the other way round.
    """
    code, lda = _rows(a, "a")
    ldb, stride = _matrices(b, "b", a.dtype)
    rows, K = a.shape
    E, N, K2 = b.shape if transB else (b.shape[0], b.shape[2], b.shape[1])
    if K != K2:
        raise ValueError(f"inner dimensions differ: {K} vs {K2}")
    off = _contiguous(offsets, "offsets", _INT32, (E + 1,))
    if out is None:
        out = _empty((rows, N), a.dtype, a.device, stream)
    _, ldo = _rows(out, "out", a.dtype)
    if tuple(out.shape) != (rows, N):
        raise ValueError("out has the wrong shape")
    _check(lib.sgemm_experts_gemm(code, int(transB), rows, N, K, E, off, a.data_ptr(), lda, b.data_ptr(), ldb, stride,
                                  out.data_ptr(), ldo, _stream_handle(stream, a, b, offsets, out)),
           "sgemm_experts_gemm")
    return out


def gemm_wgrad(a, b, offsets, out=None, *, stream=None):
    """out[e] = a_e^T @ b_e over the rows of each group: experts x M x N, zero for empty groups.

    ``a`` is rows x M, ``b`` rows x N. The gradient of :func:`gemm`'s b is ``gemm_wgrad(a, dout, offsets)``, or
    ``gemm_wgrad(dout, a, offsets)`` for ``transB``.
    """
    code, lda = _rows(a, "a")
    _, ldb = _rows(b, "b", a.dtype)
    rows, M = a.shape
    if b.shape[0] != rows:
        raise ValueError(f"a has {rows} rows, b {b.shape[0]}")
    N = b.shape[1]
    off = _contiguous(offsets, "offsets", _INT32)
    if offsets.dim() != 1 or offsets.shape[0] < 2:
        raise ValueError("offsets must be experts + 1 long")
    E = offsets.shape[0] - 1
    if out is None:
        out = _empty((E, M, N), a.dtype, a.device, stream)
    ldo, stride = _matrices(out, "out", a.dtype)
    if tuple(out.shape) != (E, M, N):
        raise ValueError("out has the wrong shape")
    _check(lib.sgemm_experts_gemm_wgrad(code, rows, M, N, E, off, a.data_ptr(), lda, b.data_ptr(), ldb,
                                        out.data_ptr(), ldo, stride, _stream_handle(stream, a, b, offsets, out)),
           "sgemm_experts_gemm_wgrad")
    return out


def w4_matvec(x, q, scales, *, group, zeros=None, ids=None, out=None, stream=None):
    """y[r, n] = sum over k of (q[e, n, k] - zero) * scale * x[r, k] with 4-bit q, a scale (and zero) per group.

    ``x`` is rows x K; ``q`` experts x N x K / 2 uint8, the even k in the low four bits; ``scales`` experts x N x
    ceil(K / group) in float32, bfloat16 or float16; ``zeros`` the same shape in uint8, or None for 8 everywhere.
    ``ids`` (rows, int32) gives each row its expert's matrix (a row without one gives zeros); without ``ids``
    there is one matrix, and ``q``, ``scales`` and ``zeros`` may be 2-D.
    """
    code, ldx = _rows(x, "x")
    rows, K = x.shape
    qp = _contiguous(q, "q", (torch.uint8,))
    if q.dim() not in (2, 3) or (q.dim() == 2 and ids is not None):
        raise ValueError("q must be experts x N x K / 2 (or N x K / 2 without ids)")
    E = q.shape[0] if q.dim() == 3 else 1
    N = q.shape[-2]
    group = int(group)
    if q.shape[-1] * 2 != K:
        raise ValueError(f"q holds {q.shape[-1] * 2} values a row, x {K}")
    if group < 1:
        raise ValueError("group must be positive")
    shape = tuple(q.shape[:-1]) + ((K + group - 1) // group,)
    sp = _contiguous(scales, "scales", tuple(TYPES), shape)
    zp = 0 if zeros is None else _contiguous(zeros, "zeros", (torch.uint8,), shape)
    ip = 0 if ids is None else _contiguous(ids, "ids", _INT32, (rows,))
    if out is None:
        out = _empty((rows, N), x.dtype, x.device, stream)
    _, ldo = _rows(out, "out", x.dtype)
    if tuple(out.shape) != (rows, N):
        raise ValueError("out has the wrong shape")
    _check(lib.sgemm_w4_matvec(code, rows, N, K, group, E, ip, x.data_ptr(), ldx, qp, sp, TYPES[scales.dtype], zp,
                               out.data_ptr(), ldo, _stream_handle(stream, x, q, scales, zeros, ids, out)),
           "sgemm_w4_matvec")
    return out

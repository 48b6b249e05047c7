"""A whole mixture-of-experts layer for a few tokens (the C ABI of include/layer.h).

Argument marshalling only, as in :mod:`dense_fp32_matrix_major_gb300.experts`, whose conventions on streams, devices,
gradients and errors this module shares. For a decoding step::

    y = layer.forward(x, ids, weights, w1, w2, gated=True)

in place of sort, gather, two products per expert, the activation and combine, which are for many tokens.
"""

from __future__ import annotations

import ctypes

import torch

from .experts import TYPES, _check, _contiguous, _empty, _rows, _stream_handle
from .fp8 import FP8_TYPES, Quantized, _blocks, _strides
from .sgemm import SGEMM_ACT_GELU, SGEMM_ACT_NONE, SGEMM_ACT_RELU, SGEMM_ACT_SILU, lib

SGEMM_LAYER_SAME = 0
SGEMM_LAYER_E4M3 = 1
SGEMM_LAYER_E5M2 = 2
SGEMM_LAYER_PAIRS_MAX = 512

ACTIVATIONS = {None: SGEMM_ACT_NONE, "none": SGEMM_ACT_NONE, "relu": SGEMM_ACT_RELU, "gelu": SGEMM_ACT_GELU,
               "silu": SGEMM_ACT_SILU}

# Every function that include/layer.h declares, with its ctypes signature.
_i64, _int, _vp, _sz = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t
SIGNATURES = {
    "sgemm_experts_layer": (_int, [_int, _int, _int, _int, _i64, _i64, _i64, _i64, _i64, _vp, _i64, _vp, _int, _vp,
                                   _vp, _i64, _i64, _vp, _vp, _i64, _i64, _vp, _vp, _i64, _vp, _sz, _vp]),
    "sgemm_experts_layer_workspace": (_sz, [_i64, _i64, _i64]),
}
for _name, (_res, _args) in SIGNATURES.items():
    _fn = getattr(lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args


def _held(w, name, dtype):
    """(how they are held, tensor, row stride, item stride, scales tensor or None) of the experts' matrices."""
    if not isinstance(w, Quantized):
        ld, stride = _strides(w, name, (dtype,), (3,))
        return SGEMM_LAYER_SAME, w, ld, stride, None
    ld, stride = _strides(w.values, name, FP8_TYPES, (3,))
    E, rows, cols = w.values.shape
    _contiguous(w.scales, f"{name}'s scales", (torch.float32,), (E, _blocks(rows), _blocks(cols)))
    return SGEMM_LAYER_E4M3 + FP8_TYPES[w.values.dtype], w.values, ld, stride, w.scales


def forward(x, ids, weights, w1, w2, *, gated=False, activation="silu", out=None, stream=None):
    """y[t] = sum over choices j of weights[t, j] * w2[e] h, e = ids[t, j], with h = activation(w1[e] x[t]), or with
    ``gated`` h = activation(a) * b of the first and second half (a, b) of w1[e] x[t].

    ``x`` is tokens x width, ``ids`` tokens x top_k int32 or int64 (an id outside 0 .. experts - 1 is left out),
    ``weights`` tokens x top_k float32, both contiguous. ``w1`` is experts x hidden x width (2 * hidden when gated) and
    ``w2`` experts x width x hidden, of x's type or 8-bit (:func:`fp8.quantize` with "blocks"). ``activation`` is
    "silu", "gelu", "relu" or None. At most SGEMM_LAYER_PAIRS_MAX pairs; for more tokens use
    :mod:`dense_fp32_matrix_major_gb300.experts`.
    """
    code, ldx = _rows(x, "x")
    tokens, width = x.shape
    if activation not in ACTIVATIONS:
        raise ValueError("activation must be silu, gelu, relu or None")
    ip = _contiguous(ids, "ids", (torch.int32, torch.int64))
    if ids.dim() != 2 or ids.shape[0] != tokens:
        raise ValueError("ids must be tokens x top_k")
    top_k = ids.shape[1]
    wp = _contiguous(weights, "weights", (torch.float32,), (tokens, top_k))
    if tokens * top_k > SGEMM_LAYER_PAIRS_MAX:
        raise ValueError(f"at most {SGEMM_LAYER_PAIRS_MAX} pairs, not {tokens * top_k}: use the experts module")
    held, m1, ld1, stride1, s1 = _held(w1, "w1", x.dtype)
    held2, m2, ld2, stride2, s2 = _held(w2, "w2", x.dtype)
    if held != held2:
        raise TypeError("w1 and w2 must be held alike")
    E, rows, cols = m1.shape
    hidden = rows // 2 if gated else rows
    if cols != width or (gated and rows % 2) or tuple(m2.shape) != (E, width, hidden):
        raise ValueError(f"w1 {tuple(m1.shape)} and w2 {tuple(m2.shape)} do not fit x {tuple(x.shape)}")
    if out is None:
        out, ldo = _empty((tokens, width), x.dtype, x.device, stream), max(width, 1)
    else:
        _, ldo = _rows(out, "out", x.dtype)
        if tuple(out.shape) != (tokens, width):
            raise ValueError("out has the wrong shape")
    need = lib.sgemm_experts_layer_workspace(tokens, top_k, hidden)
    space = _empty((need // 4,), torch.float32, x.device, stream) if need else None
    _check(lib.sgemm_experts_layer(code, held, ACTIVATIONS[activation], int(bool(gated)), tokens, top_k, E, width,
                                   hidden, x.data_ptr(), ldx, ip, 64 if ids.dtype == torch.int64 else 32, wp,
                                   m1.data_ptr(), ld1, stride1, s1.data_ptr() if s1 is not None else 0, m2.data_ptr(),
                                   ld2, stride2, s2.data_ptr() if s2 is not None else 0, out.data_ptr(), ldo,
                                   space.data_ptr() if need else 0, need,
                                   _stream_handle(stream, x, ids, weights, m1, m2, s1, s2, out)),
           "sgemm_experts_layer")
    return out

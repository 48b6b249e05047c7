"""Helpers of the tests of the 8-bit operators and of the layer for a few tokens: definitions in 64 bits and error
bounds.

Bounds are derived as in experts_harness: a sum of n products held in fp32, each addition off by at most one unit in
its last place (2^-23, rounded or cut), is off by at most (n + 1) * 2^-23 * sum |terms|; ``bound`` allows twice that,
which covers the scales' products (three roundings of 2^-24 a block). What a value is rounded to on the way adds its
half step."""

import numpy as np
import torch

from tests.experts_harness import ROUNDING, TINY, bound

E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2
LARGEST = {E4M3: 448.0, E5M2: 57344.0}
SHAPES = {"rows": (1, 128), "columns": (128, 1), "blocks": (128, 128)}


def codes(dtype):
    """The finite 8-bit values of one sign, smallest first."""
    n = 127 if dtype == E4M3 else 124
    return torch.arange(n, dtype=torch.uint8).view(dtype).double().numpy()


def quantize64(x, block, dtype, pow2=False):
    """Values and scales of a 2-D CPU tensor, block by block, from the definition."""
    high, wide = SHAPES[block]
    x = x.double().numpy()
    R, C = x.shape
    values, borders = codes(dtype), None
    borders = (values[1:] + values[:-1]) / 2
    q = np.zeros((R, C))
    scales = np.zeros((-(-R // high), -(-C // wide)), np.float32)
    for i in range(scales.shape[0]):
        for j in range(scales.shape[1]):
            at = (slice(high * i, high * (i + 1)), slice(wide * j, wide * (j + 1)))
            b = x[at]
            finite = np.abs(b[np.isfinite(b)])
            s = np.float32(finite.max() if finite.size else 0.0) / np.float32(LARGEST[dtype])
            s = max(s, np.float32(2.0 ** -126))
            if pow2:
                s = np.float32(2.0 ** np.ceil(np.log2(np.float64(s))))
            scales[i, j] = s
            with np.errstate(invalid="ignore", over="ignore"):
                y = b.astype(np.float32) * (np.float32(1) / s)
            y = np.where(np.isfinite(b), y, np.nan).astype(np.float64)
            k = np.searchsorted(borders, np.abs(y))
            tie = (k < borders.size) & (np.abs(y) == borders[np.minimum(k, borders.size - 1)]) & (k % 2 == 1)
            q[at] = np.where(np.isnan(y), np.nan, np.copysign(values[np.minimum(k + tie, values.size - 1)], y))
    return q, scales.T if block == "rows" else scales


def expand(scales, block, shape):
    """A scale for each element."""
    high, wide = SHAPES[block]
    s = scales.transpose(-1, -2) if block == "rows" else scales
    return s.repeat_interleave(high, -2).repeat_interleave(wide, -1)[..., :shape[-2], :shape[-1]]


def meaning(q, block):
    """What a Quantized stands for, in 64 bits."""
    return q.values.double() * expand(q.scales.double(), block, q.values.shape)


def check_product(got, a, b, terms, what=""):
    """got against a @ b in 64 bits, both as double tensors."""
    exact, magnitude = (a @ b).cpu().numpy(), (a.abs() @ b.abs()).cpu().numpy()
    off = np.abs(got.double().cpu().numpy() - exact)
    limit = bound(exact, magnitude, terms, got.dtype)
    bad = ~(off <= limit)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} out of bound, worst {np.nanmax(off / limit):.3g} of it"


def act64(x, act):
    if act == "silu":
        return x * torch.sigmoid(x)
    if act == "gelu":
        return x * torch.special.ndtr(x)
    return x.clamp(min=0) if act == "relu" else x


def layer64(x, ids, weights, w1, w2, gated, act):
    """The layer in 64 bits and how far a correct one may be off. w1, w2: double, experts x out x in."""
    E, F, D = w1.shape[0], w2.shape[2], x.shape[1]
    x16 = x.dtype != torch.float32
    xd = x.double()
    y, off = torch.zeros_like(xd), torch.zeros_like(xd)
    eps = 2.0 ** -23
    size = torch.zeros_like(xd)
    for e in range(E):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if not t.numel():
            continue
        pre, err = xd[t] @ w1[e].t(), 2 * (D + 2) * eps * (xd[t].abs() @ w1[e].abs().t())
        # Slopes of the activations are below 1.13; an activation is off by 2^-20 of its argument at most.
        a, ea = act64(pre[:, :F], act), 1.13 * err[:, :F] + 2.0 ** -20 * pre[:, :F].abs()
        if gated:
            b, eb = pre[:, F:], err[:, F:]
            h, eh = a * b, ea * b.abs() + a.abs() * eb + ea * eb + eps * (a * b).abs()
        else:
            h, eh = a, ea
        if x16:
            eh = eh + 2.0 ** -16 * h.abs()  # two bf16 terms
        w = weights[t, j].double()[:, None]
        out, mag = h @ w2[e].t(), h.abs() @ w2[e].abs().t()
        eo = eh @ w2[e].abs().t() + 2 * (F + 2) * eps * mag
        y.index_add_(0, t, w * out)
        size.index_add_(0, t, w.abs() * mag)
        off.index_add_(0, t, w.abs() * eo)
    off += (ids.shape[1] + 1) * eps * size
    off += ROUNDING[x.dtype] * (y.abs() + off) + TINY[x.dtype]
    return y, off


def check_layer(got, x, ids, weights, w1, w2, gated, act, what=""):
    y, off = layer64(x, ids, weights, w1, w2, gated, act)
    far = (got.double() - y).abs()
    bad = ~(far <= off)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} out of bound, worst {float((far / off).max()):.3g}"

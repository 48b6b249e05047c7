"""Cases of the 8-bit floating point operators and of the mixture-of-experts layer for a few tokens, their plain forms
and their exact values.

Three kinds of case:

* ``quantize``: a matrix in 8-bit floating point with one fp32 scale per block: 1 x 128 (``rows``, the operand of a
  product that sums along the rows), 128 x 1 (``columns``, the operand of one that sums along the columns, with
  ``experts`` > 0 in blocks that start anew with every expert's group of rows) or 128 x 128 (``blocks``, weights).
* ``product``: products of such matrices, dense (``experts`` = 0) or one per expert over its group of rows; with
  ``grad`` the gradients of the rows and of the matrices.
* ``layer``: a whole mixture-of-experts layer for a few tokens, y[t] = sum_j w[t, j] W2[e] act(W1[e] x[t]), or with
  ``gated`` W2[e] (act(G[e] x[t]) * (U[e] x[t])), G and U the halves of W1.

``run`` computes the plain form (elementary torch operations in 32 bits) or, where ``own`` is true, calls
:mod:`dense_fp32_matrix_major_gb300.fp8` and :mod:`dense_fp32_matrix_major_gb300.layer`.
"""

import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
LARGEST = {"e4m3": 448.0, "e5m2": 57344.0}
BLOCK = 128
SHAPES = {"rows": (1, BLOCK), "columns": (BLOCK, 1), "blocks": (BLOCK, BLOCK)}
TINY = 2.0 ** -126


def listed():
    return [
        # The rows of a decoding step of four sequences: latency.
        {"name": "quantize-rows-decode", "kind": "quantize", "block": "rows", "rows": 4, "width": 4096,
         "experts": 0, "type": "bf16", "to": "e4m3", "pow2": False},
        # The gradients of a large training batch in expert order, for the gradient of the experts' matrices.
        {"name": "quantize-columns-experts", "kind": "quantize", "block": "columns", "rows": 16384, "width": 2048,
         "experts": 32, "type": "bf16", "to": "e5m2", "pow2": False},
        # The fp32 master weights of sixteen experts after an update, with sides that no block divides.
        {"name": "quantize-blocks-weights", "kind": "quantize", "block": "blocks", "rows": 2049, "width": 1537,
         "experts": 16, "type": "f32", "to": "e4m3", "pow2": True},
        # A decoding step of eight sequences through one square matrix: bound by reading it.
        {"name": "product-decode", "kind": "product", "rows": 8, "n": 4096, "k": 4096, "experts": 0, "type": "bf16",
         "trans": True, "grad": False, "drop": False},
        # The forward product of a large training batch or a long prompt.
        {"name": "product-large", "kind": "product", "rows": 16384, "n": 4096, "k": 4096, "experts": 0,
         "type": "bf16", "trans": True, "grad": False, "drop": False},
        # The backward products of a batch, gradients in e5m2, those of the weights in fp32.
        {"name": "product-grad", "kind": "product", "rows": 8192, "n": 4096, "k": 2048, "experts": 0, "type": "bf16",
         "trans": True, "grad": True, "drop": False},
        # A layer's forward product over many experts.
        {"name": "product-experts", "kind": "product", "rows": 16384, "n": 4096, "k": 2048, "experts": 32,
         "type": "bf16", "trans": True, "grad": False, "drop": False},
        # The backward products of a ragged micro-batch, dropped rows, matrices stored the other way round.
        {"name": "product-experts-grad", "kind": "product", "rows": 4093, "n": 1024, "k": 2048, "experts": 16,
         "type": "f16", "trans": False, "grad": True, "drop": True},
        # One token through eight of 64 fine-grained experts.
        {"name": "layer-single", "kind": "layer", "tokens": 1, "top_k": 8, "experts": 64, "width": 2048,
         "hidden": 1024, "type": "bf16", "weights": "same", "gated": True, "act": "silu", "drop": False},
        # A decoding batch of eight sequences from 8-bit experts.
        {"name": "layer-fp8", "kind": "layer", "tokens": 8, "top_k": 2, "experts": 16, "width": 4096,
         "hidden": 4096, "type": "bf16", "weights": "fp8", "gated": True, "act": "silu", "drop": False},
        # Three tokens in fp32 with widths whose rows are not 16-byte aligned, without a gate.
        {"name": "layer-f32-odd", "kind": "layer", "tokens": 3, "top_k": 4, "experts": 32, "width": 1537,
         "hidden": 1023, "type": "f32", "weights": "same", "gated": False, "act": "gelu", "drop": True},
        # Thirty-two tokens that between them reach most of 128 small experts.
        {"name": "layer-batch", "kind": "layer", "tokens": 32, "top_k": 8, "experts": 128, "width": 2048,
         "hidden": 768, "type": "f16", "weights": "same", "gated": True, "act": "silu", "drop": False},
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def _size(rng, lo, hi):
    """A size between lo and hi: a multiple of 64, or now and then any number."""
    return _log(rng, lo, hi) if rng.random() < 0.3 else max(lo, _log(rng, lo, hi) // 64 * 64)


def draw(rng):
    kind = rng.choice(["quantize", "product", "product", "layer"])
    c = {"kind": kind, "type": rng.choice(["f32", "bf16", "f16"])}
    if kind == "quantize":
        c["block"] = rng.choice(["rows", "columns", "blocks"])
        c["experts"] = rng.choice([0, 0, 4, 16, 64])
        if c["block"] == "rows":
            c["experts"] = 0
        c["width"] = _size(rng, 64, 4096)
        most = 16384 * 4096 // c["width"] // (max(c["experts"], 1) if c["block"] == "blocks" else 1)
        c["rows"] = _log(rng, 1, min(most, 32768))
        c["to"] = rng.choice(["e4m3", "e4m3", "e5m2"])
        c["pow2"] = rng.random() < 0.4
    elif kind == "product":
        c["experts"] = rng.choice([0, 0, 0, 1, 4, 8, 32, 64])
        c["n"] = _size(rng, 64, 4096)
        c["k"] = _size(rng, 64, 4096 if c["experts"] < 32 else 2048)
        c["grad"] = rng.random() < 0.4
        c["rows"] = _log(rng, 1, min(32768, 16384 * 4096 * 4096 // (c["n"] * c["k"]) // (2 if c["grad"] else 1)))
        c["trans"] = rng.random() < 0.6
        c["drop"] = c["experts"] > 0 and rng.random() < 0.4
    else:
        c["tokens"] = _log(rng, 1, 64)
        c["top_k"] = rng.choice([1, 2, 2, 4, 6, 8])
        c["experts"] = rng.choice([8, 16, 32, 60, 64, 128])
        c["weights"] = rng.choice(["same", "same", "fp8"])
        c["gated"] = rng.random() < 0.7
        c["act"] = rng.choice(["silu", "silu", "gelu", "relu"])
        c["drop"] = rng.random() < 0.3
        most = 128 * 2048 * 768 * 2 // c["experts"]
        most = min(most, 256 * 2048 * 768 * 2 // (c["tokens"] * c["top_k"]))
        most = most // BYTES[c["type"]]
        c["width"] = _size(rng, 64, min(4096, most // 64))
        c["hidden"] = _size(rng, 64, max(64, min(4096, most // c["width"])))
    return c


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(g, shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _activations(g, shape, dtype):
    """Rows as a layer gives them: a few channels and rows are much larger than the rest."""
    x = torch.randn(shape, generator=g, device="cuda")
    for dim in (-1, -2):
        size = [1] * len(shape)
        size[dim] = shape[dim]
        x *= torch.exp(0.7 * torch.randn(size, generator=g, device="cuda"))
    return x.to(dtype)


def _offsets(rows, experts, drop, g):
    p = torch.softmax(0.5 * torch.randn(experts, generator=g, device="cuda"), 0)
    if drop:
        p = torch.cat([p, torch.tensor([0.03], device="cuda")])
    expert = torch.multinomial(p, rows, replacement=True, generator=g)
    counts = torch.bincount(expert, minlength=experts)[:experts]
    return torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32), int(counts.max())


def _choices(case, g):
    T, k, E = case["tokens"], case["top_k"], case["experts"]
    scores = torch.randn((T, E), generator=g, device="cuda") + 0.5 * torch.randn((1, E), generator=g, device="cuda")
    top, ids = scores.topk(k, dim=1)
    weights = torch.softmax(top, dim=1).contiguous()
    if case["drop"]:
        ids = torch.where(torch.rand((T, k), generator=g, device="cuda") < 0.05, -1, ids)
    return ids.contiguous(), weights


def _aligned(q):
    """The same matrices in rows that start 16 bytes apart (a product's operands)."""
    width = q.shape[-1]
    store = torch.zeros((*q.shape[:-1], -(-width // 16) * 16), dtype=torch.uint8, device=q.device).view(q.dtype)
    store.view(torch.uint8)[..., :width] = q.view(torch.uint8)
    return store[..., :width]


def _handy(x, block, to):
    """8-bit operands a program has in hand: values and scales of x, rounded once by PyTorch."""
    high, wide = SHAPES[block]
    R, C = x.shape[-2:]
    blocks = _cut(x.float(), high, wide)
    scale = (blocks.abs().amax((-3, -1)) / LARGEST[to]).clamp(min=TINY)
    q = (blocks / scale[..., :, None, :, None]).clamp(-LARGEST[to], LARGEST[to])
    q = q.reshape(*x.shape[:-2], -(-R // high) * high, -(-C // wide) * wide)[..., :R, :C].to(FP8[to])
    return _aligned(q), (scale.transpose(-1, -2) if block == "rows" else scale).contiguous()


def prepare(case, seed):
    g = _gen(seed)
    dt = TYPES[case["type"]]
    s = dict(case)
    if case["kind"] == "quantize":
        R, C, E = case["rows"], case["width"], case["experts"]
        if case["block"] == "blocks":
            s["x"] = _normal(g, (E, R, C) if E else (R, C), dt, 0.02)
        else:
            s["x"] = _activations(g, (R, C), dt)
        s["offsets"] = _offsets(R, E, False, g)[0] if E and case["block"] == "columns" else None
    elif case["kind"] == "product":
        S, N, K, E = case["rows"], case["n"], case["k"], case["experts"]
        s["offsets"], s["most"] = _offsets(S, E, case["drop"], g) if E else (None, S)
        shape = (N, K) if case["trans"] else (K, N)
        s["w"] = _handy(_normal(g, (E, *shape) if E else shape, scale=K ** -0.5), "blocks", "e4m3")
        x = _activations(g, (S, K), torch.bfloat16)
        if case["grad"]:
            # The same rows as both products read them: scaled along the row, and along the column of each group.
            dy = _activations(g, (S, N), torch.bfloat16)
            s["dy_rows"] = _handy(dy, "rows", "e5m2")
            s["dy"] = _handy(_blocks_of_groups(dy, s["offsets"]), "columns", "e5m2")
            s["x"] = _handy(_blocks_of_groups(x, s["offsets"]), "columns", "e4m3")
        else:
            s["x"] = _handy(x, "rows", "e4m3")
    else:
        T, E, D, F = case["tokens"], case["experts"], case["width"], case["hidden"]
        s["ids"], s["weights_of"] = _choices(case, g)
        s["x"] = _normal(g, (T, D), dt)
        for name, shape in (("w1", (E, F * (2 if case["gated"] else 1), D)), ("w2", (E, D, F))):
            if case["weights"] == "fp8":
                q = (100 * torch.randn(shape, generator=g, device="cuda")).clamp_(-448, 448).to(FP8["e4m3"])
                n = [-(-i // BLOCK) for i in shape[1:]]
                scale = 0.5 + torch.rand((E, *n), generator=g, device="cuda")
                s[name] = (_aligned(q), scale * (0.01 * shape[2] ** -0.5))
            else:
                s[name] = _normal(g, shape, dt, shape[2] ** -0.5)
    return s


def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    if s["kind"] == "layer":
        from dense_fp32_matrix_major_gb300 import fp8, layer

        w1, w2 = s["w1"], s["w2"]
        if s["weights"] == "fp8":
            w1, w2 = fp8.Quantized(*w1), fp8.Quantized(*w2)
        return {"y": layer.forward(s["x"], s["ids"], s["weights_of"], w1, w2, gated=s["gated"], activation=s["act"])}
    from dense_fp32_matrix_major_gb300 import fp8

    if s["kind"] == "quantize":
        q = fp8.quantize(s["x"], s["block"], dtype=FP8[s["to"]], pow2=s["pow2"], offsets=s["offsets"])
        return {"q": q.values, "scales": q.scales}
    dt, w = TYPES[s["type"]], fp8.Quantized(*s["w"])
    if not s["grad"]:
        return {"y": fp8.gemm(fp8.Quantized(*s["x"]), w, s["offsets"], transB=s["trans"], dtype=dt)}
    dx = fp8.gemm(fp8.Quantized(*s["dy_rows"]), w, s["offsets"], transB=not s["trans"], dtype=dt)
    left, right = (s["dy"], s["x"]) if s["trans"] else (s["x"], s["dy"])
    dw = fp8.gemm_wgrad(fp8.Quantized(*left), fp8.Quantized(*right), s["offsets"], dtype=torch.float32)
    return {"dx": dx, "dw": dw}


def _cut(x, high, wide):
    """x with its last two dimensions in blocks (..., block row, row, block column, column), zeros past the end."""
    R, C = x.shape[-2:]
    x = torch.nn.functional.pad(x, (0, -C % wide, 0, -R % high))
    return x.unflatten(-1, (-1, wide)).unflatten(-3, (-1, high))


def _block_rows(offsets, rows):
    """The row of x in each row of the groups' blocks of 128 rows; `rows` where the block has none."""
    counts = (offsets[1:] - offsets[:-1]).long()
    ends = ((counts + BLOCK - 1) // BLOCK).cumsum(0)
    E = counts.numel()
    b = torch.arange((rows + (BLOCK - 1) * min(E, rows)) // BLOCK, device=offsets.device)
    e = torch.searchsorted(ends, b, right=True)
    within = (b - torch.where(e > 0, ends[(e - 1).clamp(min=0)], 0))[:, None] * BLOCK
    within = within + torch.arange(BLOCK, device=b.device)
    e = e.clamp(max=E - 1)[:, None]
    used = (b < ends[-1])[:, None] & (within < counts[e])
    return torch.where(used, offsets[e] + within, rows).reshape(-1)


def _blocks_of_groups(x, offsets):
    """x with every group's rows in whole blocks of 128, zeros where a group has no row."""
    if offsets is None:
        return x
    return torch.cat([x, x.new_zeros(1, x.shape[1])])[_block_rows(offsets, x.shape[0])]


def _nearest(y, to):
    """The 8-bit value nearest to y (in 64 bits), ties to even."""
    digits, low = (3, -6) if to == "e4m3" else (2, -14)
    e = (torch.frexp(y).exponent - 1).clamp(low, 16).long()
    step = torch.tensor([2.0 ** i for i in range(-20, 17)], dtype=torch.float64, device=y.device)[e - digits + 20]
    q = (torch.round(y / step) * step).clamp(-LARGEST[to], LARGEST[to])
    return q.to(torch.float32).to(FP8[to])


def _quantized(x, block, to, pow2):
    """Plain form of the quantisation: the values and their scales."""
    high, wide = SHAPES[block]
    R, C = x.shape[-2:]
    b = _cut(x.float(), high, wide)
    finite = torch.isfinite(b)
    # A divisor on the device: PyTorch multiplies by the reciprocal of a plain number.
    largest = torch.full((1,), LARGEST[to], device=x.device)
    scale = (torch.where(finite, b.abs(), 0.0).amax((-3, -1)) / largest).clamp(min=TINY)
    if pow2:
        mantissa, e = torch.frexp(scale)
        scale = torch.ldexp(torch.ones_like(scale), torch.where(mantissa == 0.5, e - 1, e))
    # As defined: the product with the scale's reciprocal, both in fp32, then the nearest 8-bit value.
    y = (torch.where(finite, b, float("nan")) * torch.reciprocal(scale)[..., :, None, :, None]).double()
    y = y.reshape(*x.shape[:-2], -(-R // high) * high, -(-C // wide) * wide)[..., :R, :C]
    q = torch.where(torch.isnan(y), float("nan"), _nearest(torch.nan_to_num(y), to).float()).to(FP8[to])
    return q, (scale.transpose(-1, -2) if block == "rows" else scale).contiguous()


def _values(q, scales, block):
    """What quantised values stand for, in 32 bits."""
    high, wide = SHAPES[block]
    s = scales.transpose(-1, -2) if block == "rows" else scales
    s = s.repeat_interleave(high, -2) if high > 1 else s
    s = s.repeat_interleave(wide, -1) if wide > 1 else s
    return q.float() * s[..., :q.shape[-2], :q.shape[-1]]


def _padded(x, offsets, most):
    """The rows of each group as (experts, most, width) in 32 bits, zero past the group's end."""
    at = offsets[:-1, None].long() + torch.arange(most, device=x.device)
    inside = at < offsets[1:, None]
    return torch.where(inside[..., None], x[at.clamp(max=x.shape[0] - 1)], 0.0)


def _unpadded(p, offsets, rows):
    """The groups of p back in their rows; zero for rows outside every group."""
    row = torch.arange(rows, device=p.device)
    e = torch.searchsorted(offsets, row.to(torch.int32), right=True) - 1
    inside = e < p.shape[0]
    e = e.clamp(max=p.shape[0] - 1)
    at = (row - offsets[e]).clamp(max=p.shape[1] - 1)
    return torch.where(inside[:, None], p[e, at], 0.0)


def _group_blocks(x, offsets, most):
    """The blocks of each group as (experts, rows, width), zero past the group's end."""
    blocks = ((offsets[1:] - offsets[:-1]).long() + BLOCK - 1) // BLOCK
    first = (blocks.cumsum(0) - blocks) * BLOCK
    within = torch.arange(-(-max(most, 1) // BLOCK) * BLOCK, device=x.device)
    at = (first[:, None] + within).clamp(max=x.shape[0] - 1)
    return torch.where((within < blocks[:, None] * BLOCK)[..., None], x[at], 0.0)


def _act(x, act):
    if act == "silu":
        return x / (1 + torch.exp(-x))
    if act == "gelu":
        return 0.5 * x * (1 + torch.erf(x * math.sqrt(0.5)))
    return torch.where(x < 0, 0.0, x)


def _run_plain(s):
    dt = TYPES[s["type"]]
    if s["kind"] == "quantize":
        q, scales = _quantized(_blocks_of_groups(s["x"], s["offsets"]), s["block"], s["to"], s["pow2"])
        return {"q": q, "scales": scales}
    if s["kind"] == "product":
        w = _values(*s["w"], "blocks")
        w = w if s["trans"] else w.transpose(-1, -2)  # n x k
        if not s["grad"]:
            x = _values(*s["x"], "rows")
            if s["offsets"] is None:
                return {"y": (x @ w.t()).to(dt)}
            y = torch.bmm(_padded(x, s["offsets"], s["most"]), w.transpose(1, 2))
            return {"y": _unpadded(y, s["offsets"], s["rows"]).to(dt)}
        left, right = _values(*s["dy"], "columns"), _values(*s["x"], "columns")
        if not s["trans"]:
            left, right = right, left
        dy = _values(*s["dy_rows"], "rows")
        if s["offsets"] is None:
            return {"dx": (dy @ w).to(dt), "dw": left.t() @ right}
        dx = torch.bmm(_padded(dy, s["offsets"], s["most"]), w)
        dw = torch.bmm(_group_blocks(left, s["offsets"], s["most"]).transpose(1, 2),
                       _group_blocks(right, s["offsets"], s["most"]))
        return {"dx": _unpadded(dx, s["offsets"], s["rows"]).to(dt), "dw": dw}
    T, k, F = s["tokens"], s["top_k"], s["hidden"]
    ids = s["ids"].reshape(-1)
    kept, at = ids >= 0, ids.clamp(min=0)
    rows = s["x"].float().repeat_interleave(k, 0)
    w1, w2 = ((_values(w[0][at], w[1][at], "blocks") if s["weights"] == "fp8" else w[at].float())
              for w in (s["w1"], s["w2"]))
    h = torch.bmm(w1, rows[:, :, None])[..., 0]
    h = _act(h[:, :F], s["act"]) * h[:, F:] if s["gated"] else _act(h, s["act"])
    y = torch.bmm(w2, h[:, :, None])[..., 0]
    y = torch.where(kept[:, None], y * s["weights_of"].reshape(-1, 1), 0.0)
    return {"y": y.reshape(T, k, -1).sum(1).to(dt)}


def work(case):
    b = BYTES[case["type"]]
    if case["kind"] == "quantize":
        E = case["experts"]
        n = case["rows"] * case["width"] * (max(E, 1) if case["block"] == "blocks" else 1)
        high, wide = SHAPES[case["block"]]
        return {"bytes": n * (b + 1) + 4 * n // (high * wide), "flops": 2 * n}
    if case["kind"] == "product":
        S, N, K, E = case["rows"], case["n"], case["k"], case["experts"]
        weights = (min(E, S) if E else 1) * N * K
        if not case["grad"]:
            return {"bytes": int(S * K * (1 + 4 / BLOCK)) + weights + S * N * b, "flops": 2 * S * N * K}
        read = (2 * S * N + S * K) * (1 + 4 / BLOCK) + weights
        return {"bytes": int(read + S * K * b + max(E, 1) * N * K * 4), "flops": 4 * S * N * K}
    T, k, E, D, F = (case[i] for i in ("tokens", "top_k", "experts", "width", "hidden"))
    used = E * (1 - (1 - k / E) ** T) if k < E else E  # experts that T tokens with k distinct choices reach
    per = (3 if case["gated"] else 2) * F * D
    return {"bytes": int(used * per * (1 if case["weights"] == "fp8" else b) + 2 * T * D * b), "flops": 2 * T * k * per}


def _exact_codes(x, scale, to):
    """The 8-bit values nearest to fp32(x * fp32(1 / scale)) by a search among all of them, ties to the even code."""
    codes = torch.arange(127 if to == "e4m3" else 124, dtype=torch.uint8, device=x.device)
    values = codes.view(FP8[to]).double()
    borders = (values[1:] + values[:-1]) / 2
    y = (x.double() * (1 / scale.double()).float().double()).float().double().abs()
    at = torch.bucketize(y, borders)
    tie = (at < borders.numel()) & (y == borders[at.clamp(max=borders.numel() - 1)]) & (at % 2 == 1)
    return torch.copysign(values[at + tie], x.double())


def _exact_sum(a, sa, b, sb):
    """a b^T summed block of 128 by block, each scaled in 64 bits; sa, sb: (blocks, rows of a / b) or broadcast."""
    out = torch.zeros((a.shape[0], b.shape[0]), dtype=torch.float64, device=a.device)
    for i in range(-(-a.shape[1] // BLOCK)):
        k = slice(BLOCK * i, BLOCK * (i + 1))
        out += (a[:, k].double() * sa[i].double()[:, None]) @ (b[:, k].double() * sb[i].double()[:, None]).t()
    return out


def _exact_rows(a, sa, w, sw):
    """Rows (scaled 1 x 128) times a matrix n x k (scaled 128 x 128), both as 8-bit values."""
    per_row = sw.repeat_interleave(BLOCK, 0)[:w.shape[0]]  # n x blocks of k
    return _exact_sum(a, sa, w, per_row.t())


def exact(case, seed):
    """The same outputs in 64 bits, from the definitions, one block or expert at a time."""
    s = prepare(case, seed)
    if case["kind"] == "quantize":
        x, (high, wide), to = s["x"], SHAPES[case["block"]], case["to"]
        if s["offsets"] is not None:
            off, R = s["offsets"].tolist(), case["rows"]
            parts = []
            for e in range(case["experts"]):
                part = x[off[e]:off[e + 1]]
                parts += [part, part.new_zeros(-part.shape[0] % BLOCK, x.shape[1])]
            used = sum(p.shape[0] for p in parts)
            total = (R + (BLOCK - 1) * min(case["experts"], R)) // BLOCK * BLOCK
            x = torch.cat([*parts, x.new_zeros(total - used, x.shape[1])])
        x = x[None] if x.dim() == 2 else x
        qs, scales = [], []
        for m in x:
            R, C = m.shape
            most = m.abs().double()
            most = torch.cat([most, most.new_zeros(-R % high, C)]).reshape(-1, high, C).amax(1)
            most = torch.cat([most, most.new_zeros(most.shape[0], -C % wide)], 1)
            most = most.reshape(most.shape[0], -1, wide).amax(2)
            scale = (most / LARGEST[to]).clamp(min=TINY)
            held = scale.float()
            if case["pow2"]:
                scale = torch.tensor([[2.0 ** math.ceil(math.log2(v)) for v in r] for r in held.tolist()],
                                     dtype=torch.float64, device=m.device)
                held = scale.float()
            at_r, at_c = torch.arange(R, device=m.device) // high, torch.arange(C, device=m.device) // wide
            qs.append(_exact_codes(m, held[at_r][:, at_c], to))
            scales.append(scale.t() if case["block"] == "rows" else scale)
        q, scale = torch.stack(qs), torch.stack(scales)
        return {"q": q if s["x"].dim() == 3 else q[0], "scales": scale if s["x"].dim() == 3 else scale[0]}
    if case["kind"] == "product":
        S, N, K, E = case["rows"], case["n"], case["k"], case["experts"]
        off = s["offsets"].tolist() if E else [0, S]
        w, sw = (t if E else t[None] for t in s["w"])
        if not case["trans"]:
            w, sw = w.view(torch.uint8).transpose(1, 2).contiguous().view(w.dtype), sw.transpose(1, 2)
        if not case["grad"]:
            x, sx = s["x"]
            y = torch.zeros((S, N), dtype=torch.float64, device="cuda")
            for e in range(max(E, 1)):
                r = slice(off[e], off[e + 1])
                y[r] = _exact_rows(x[r], sx[:, r], w[e], sw[e])
            return {"y": y}
        dy, sdy = s["dy_rows"]
        dx = torch.zeros((S, K), dtype=torch.float64, device="cuda")
        dw = torch.zeros((max(E, 1), N, K), dtype=torch.float64, device="cuda")
        block = 0
        for e in range(max(E, 1)):
            r = slice(off[e], off[e + 1])
            wt = w[e].view(torch.uint8).t().contiguous().view(w.dtype)
            dx[r] = _exact_rows(dy[r], sdy[:, r], wt, sw[e].t())
            blocks = -(-(off[e + 1] - off[e]) // BLOCK)
            rows, b = slice(block * BLOCK, (block + blocks) * BLOCK), slice(block, block + blocks)
            left, right = (t[0].view(torch.uint8)[rows].t().contiguous().view(t[0].dtype) for t in (s["dy"], s["x"]))
            dw[e] = _exact_sum(left, s["dy"][1][b], right, s["x"][1][b])
            block += blocks
        dw = dw if case["trans"] else dw.transpose(1, 2).contiguous()
        return {"dx": dx, "dw": dw if E else dw[0]}
    y = torch.zeros((case["tokens"], case["width"]), dtype=torch.float64, device="cuda")
    F = case["hidden"]

    def matrix(w, e):
        if case["weights"] != "fp8":
            return w[e].double()
        r, c = (torch.arange(n, device="cuda") // BLOCK for n in w[0].shape[1:])
        return w[0][e].double() * w[1][e].double()[r][:, c]

    for e in sorted(set(s["ids"].reshape(-1).tolist()) - {-1}):
        t, j = torch.nonzero(s["ids"] == e, as_tuple=True)
        h = s["x"][t].double() @ matrix(s["w1"], e).t()
        gate = h[:, :F]
        if case["act"] == "silu":
            gate = gate * torch.sigmoid(gate)
        elif case["act"] == "gelu":
            gate = gate * torch.special.ndtr(gate)
        else:
            gate = gate.clamp(min=0)
        h = gate * h[:, F:] if case["gated"] else gate
        y.index_add_(0, t, (h @ matrix(s["w2"], e).t()) * s["weights_of"][t, j].double()[:, None])
    return {"y": y}

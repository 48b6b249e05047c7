"""Cases of the operators of a mixture-of-experts layer, their plain forms and their exact values.

Four kinds of case:

* ``dispatch``: (token, choice) pairs sorted by expert, and the tokens' rows gathered in that order; with
  ``grad`` also the gather's gradient.
* ``combine``: the experts' rows weighted and summed back per token; with ``grad`` also the gradients of the
  rows and of the weights.
* ``gemm``: one product per expert over its group of rows; with ``grad`` the gradients of the rows and of the
  experts' matrices.
* ``w4``: matrix-vector products with 4-bit weights and group scales, one matrix for all rows (``experts`` = 1)
  or each row with the matrix of its expert.

``run`` computes the plain form (elementary torch operations in 32 bits) or, where ``own`` is true, calls
:mod:`dense_fp32_matrix_major_gb300.experts`.
"""

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}


def listed():
    return [
        # A decoding step of four sequences: latency of the sort and the row copies.
        {"name": "dispatch-decode", "kind": "dispatch", "tokens": 4, "top_k": 2, "experts": 8, "width": 1024,
         "type": "bf16", "ids": "int64", "drop": False, "grad": False},
        # A training step's micro-batch in fp32, some choices dropped by a capacity limit, forward and backward.
        {"name": "dispatch-train", "kind": "dispatch", "tokens": 4096, "top_k": 2, "experts": 16, "width": 2048,
         "type": "f32", "ids": "int32", "drop": True, "grad": True},
        # A large prefill or training batch over many fine-grained experts.
        {"name": "dispatch-large", "kind": "dispatch", "tokens": 16384, "top_k": 8, "experts": 128, "width": 2048,
         "type": "bf16", "ids": "int64", "drop": False, "grad": False},
        # A decoding step of three sequences with a width whose rows are not 16-byte aligned.
        {"name": "combine-decode-odd", "kind": "combine", "tokens": 3, "top_k": 4, "experts": 32, "width": 1537,
         "type": "f32", "ids": "int32", "drop": False, "grad": False},
        # A large training batch, forward and both gradients.
        {"name": "combine-train-large", "kind": "combine", "tokens": 16384, "top_k": 8, "experts": 64,
         "width": 2048, "type": "bf16", "ids": "int32", "drop": True, "grad": True},
        # A layer's forward product in the library's own precision, eight experts.
        {"name": "gemm-f32", "kind": "gemm", "rows": 8192, "experts": 8, "k": 1024, "n": 2048, "type": "f32",
         "trans": False, "drop": False, "grad": False},
        # The backward products of a ragged micro-batch in fp32, matrices stored transposed, dropped rows.
        {"name": "gemm-f32-grad-ragged", "kind": "gemm", "rows": 4093, "experts": 16, "k": 2048, "n": 1024,
         "type": "f32", "trans": True, "drop": True, "grad": True},
        # A decoding batch: a few rows per expert, bound by reading the experts' matrices.
        {"name": "gemm-bf16-few-rows", "kind": "gemm", "rows": 64, "experts": 32, "k": 2048, "n": 2048,
         "type": "bf16", "trans": True, "drop": False, "grad": False},
        # The backward products of a large batch in bf16.
        {"name": "gemm-bf16-grad-large", "kind": "gemm", "rows": 16384, "experts": 32, "k": 2048, "n": 4096,
         "type": "bf16", "trans": True, "drop": False, "grad": True},
        # One token through one quantised square matrix.
        {"name": "w4-single", "kind": "w4", "rows": 1, "experts": 1, "k": 4096, "n": 4096, "group": 128,
         "type": "bf16", "zeros": False},
        # Eight tokens with two experts each, quantised experts with zero points.
        {"name": "w4-experts", "kind": "w4", "rows": 16, "experts": 16, "k": 2048, "n": 4096, "group": 64,
         "type": "f16", "zeros": True},
        # Eight tokens in fp32 through a large quantised matrix.
        {"name": "w4-wide", "kind": "w4", "rows": 8, "experts": 1, "k": 8192, "n": 16384, "group": 128,
         "type": "f32", "zeros": True},
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    kind = rng.choice(["dispatch", "combine", "gemm", "w4"])
    c = {"kind": kind, "type": rng.choice(["f32", "bf16", "f16"])}
    if kind in ("dispatch", "combine"):
        c["experts"] = rng.choice([4, 7, 8, 16, 32, 60, 64, 128, 160, 256])
        c["top_k"] = min(rng.choice([1, 2, 2, 3, 4, 6, 8]), c["experts"])
        c["width"] = _log(rng, 64, 3000) if rng.random() < 0.35 else 64 * _log(rng, 1, 40)
        size = 4 if c["type"] == "f32" else 2
        c["tokens"] = _log(rng, 1, min(65536, 16384 * 9 * 2048 * 2 // ((c["top_k"] + 1) * c["width"] * size)))
        c["ids"] = rng.choice(["int32", "int64"])
        c["drop"] = rng.random() < 0.4
        c["grad"] = rng.random() < 0.5
    elif kind == "gemm":
        c["experts"] = rng.choice([1, 2, 5, 8, 16, 32, 64, 128])
        odd = rng.random() < 0.25
        c["k"] = _log(rng, 33, 3000) if odd else 64 * _log(rng, 2, 40)
        most = max(64, min(2560, 32 * 2048 * 4096 // (c["experts"] * c["k"])))
        c["n"] = _log(rng, 33, most) if odd else 64 * _log(rng, 1, most // 64)
        c["grad"] = rng.random() < 0.4
        work = 16384 * 2048 * 4096 * 2 // (2 if c["grad"] else 1)
        # An fp32 product has an eighth of the multiply-adds of the largest 16-bit one.
        work //= 8 if c["type"] == "f32" else 1
        c["rows"] = _log(rng, 1, max(1, min(32768, work // (c["k"] * c["n"]))))
        c["trans"] = rng.random() < 0.5
        c["drop"] = rng.random() < 0.3
    else:
        c["experts"] = rng.choice([1, 1, 1, 4, 8, 32])
        c["group"] = rng.choice([32, 64, 128, 128])
        c["k"] = c["group"] * max(1, _log(rng, 64, 8192) // c["group"])
        c["k"] += c["group"] if c["k"] == 3072 else 0
        c["rows"] = _log(rng, 1, 16)
        used = min(c["experts"], c["rows"])
        c["n"] = _log(rng, 64, min(28672, 16384 * 8192 // (c["k"] * used)))
        c["zeros"] = rng.random() < 0.5
    return c


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _choices(case, g):
    """Expert choices (distinct per token, some experts more popular than others) and their weights."""
    T, k, E = case["tokens"], case["top_k"], case["experts"]
    scores = torch.randn((T, E), generator=g, device="cuda") + torch.randn((1, E), generator=g, device="cuda")
    top, ids = scores.topk(k, dim=1)
    weights = torch.softmax(top, dim=1).contiguous()
    if case["drop"]:
        ids = torch.where(torch.rand((T, k), generator=g, device="cuda") < 0.05, -1, ids)
    return ids.to(torch.int64 if case["ids"] == "int64" else torch.int32).contiguous(), weights


def _sorted_pairs(ids, experts):
    """offsets, order and slot of the pairs sorted by expert, pairs without an expert last."""
    flat = ids.reshape(-1)
    key = torch.where((flat < 0) | (flat >= experts), experts, flat.to(torch.int64))
    order = torch.argsort(key, stable=True)
    slot = torch.empty_like(order)
    slot[order] = torch.arange(order.numel(), device=order.device)
    offsets = torch.searchsorted(key[order], torch.arange(experts + 1, device=key.device))
    return offsets.to(torch.int32), order.to(torch.int32), slot.to(torch.int32).reshape(ids.shape)


def _group_offsets(case, g):
    S, E = case["rows"], case["experts"]
    p = torch.softmax(0.5 * torch.randn(E, generator=g, device="cuda"), 0)
    if case["drop"]:
        p = torch.cat([p, torch.tensor([0.03], device="cuda")])
    expert = torch.multinomial(p, S, replacement=True, generator=g)
    counts = torch.bincount(expert, minlength=E)[:E]
    return torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32), int(counts.max())


def prepare(case, seed):
    g = _gen(seed)
    dt = TYPES[case["type"]]
    s = dict(case)
    if case["kind"] == "dispatch":
        s["ids"], _ = _choices(case, g)
        s["x"] = _normal(g, (case["tokens"], case["width"]), dt)
        if case["grad"]:
            s["dxs"] = _normal(g, (case["tokens"] * case["top_k"], case["width"]), dt)
    elif case["kind"] == "combine":
        ids, s["weights"] = _choices(case, g)
        s["offsets"], s["order"], s["slot"] = _sorted_pairs(ids, case["experts"])
        s["h"] = _normal(g, (case["tokens"] * case["top_k"], case["width"]), dt)
        if case["grad"]:
            s["dy"] = _normal(g, (case["tokens"], case["width"]), dt)
    elif case["kind"] == "gemm":
        E, K, N, S = case["experts"], case["k"], case["n"], case["rows"]
        # The most rows of one expert: a program that pads its groups knows it (its capacity).
        s["offsets"], s["most"] = _group_offsets(case, g)
        s["a"] = _normal(g, (S, K), dt)
        s["b"] = _normal(g, (E, N, K) if case["trans"] else (E, K, N), dt, K ** -0.5)
        if case["grad"]:
            s["dc"] = _normal(g, (S, N), dt)
    else:
        E, K, N, G, R = case["experts"], case["k"], case["n"], case["group"], case["rows"]
        s["x"] = _normal(g, (R, K), dt)
        s["q"] = torch.randint(0, 256, (E, N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
        s["scales"] = ((torch.rand((E, N, K // G), generator=g, device="cuda") + 0.5) * (0.1 * K ** -0.5)).to(dt)
        s["zeros"] = (torch.randint(0, 16, (E, N, K // G), generator=g, device="cuda", dtype=torch.uint8)
                      if case["zeros"] else None)
        s["ids"] = (torch.randint(0, E, (R,), generator=g, device="cuda", dtype=torch.int32) if E > 1 else None)
    return s


def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    from dense_fp32_matrix_major_gb300 import experts

    if s["kind"] == "dispatch":
        r = experts.sort(s["ids"], s["experts"])
        out = {"offsets": r.offsets, "order": r.order, "slot": r.slot, "xs": experts.gather(s["x"], r)}
        if s["grad"]:
            out["dx"] = experts.gather_grad(s["dxs"], r)
        return out
    if s["kind"] == "combine":
        r = experts.Routing(s["offsets"], s["order"], s["slot"])
        out = {"y": experts.combine(s["h"], s["weights"], r)}
        if s["grad"]:
            out["dh"], out["dw"] = experts.combine_grad(s["dy"], s["h"], s["weights"], r)
        return out
    if s["kind"] == "gemm":
        if not s["grad"]:
            return {"c": experts.gemm(s["a"], s["b"], s["offsets"], transB=s["trans"])}
        da = experts.gemm(s["dc"], s["b"], s["offsets"], transB=not s["trans"])
        left, right = (s["dc"], s["a"]) if s["trans"] else (s["a"], s["dc"])
        return {"da": da, "db": experts.gemm_wgrad(left, right, s["offsets"])}
    return {"y": experts.w4_matvec(s["x"], s["q"], s["scales"], zeros=s["zeros"], group=s["group"], ids=s["ids"])}


def _rows_of_pairs(rows, slot, kept):
    """rows[slot] as (tokens, top_k, width) in 32 bits, zero for pairs that were dropped."""
    return torch.where(kept[..., None], rows[slot.long()].float(), 0.0)


def _padded(x, offsets, most):
    """The rows of each group as (experts, most, width) in 32 bits, zero past the group's end."""
    at = offsets[:-1, None].long() + torch.arange(most, device=x.device)
    inside = at < offsets[1:, None]
    return torch.where(inside[..., None], x[at.clamp(max=x.shape[0] - 1)].float(), 0.0)


def _unpadded(p, offsets, rows):
    """The groups of p back in their rows; zero for rows outside every group."""
    row = torch.arange(rows, device=p.device)
    e = torch.searchsorted(offsets, row.to(torch.int32), right=True) - 1
    inside = e < p.shape[0]
    e = e.clamp(max=p.shape[0] - 1)
    at = (row - offsets[e]).clamp(max=p.shape[1] - 1)
    return torch.where(inside[:, None], p[e, at], 0.0)


def _nibbles(q):
    return torch.stack([q & 15, q >> 4], dim=-1).flatten(-2)


def _run_plain(s):
    dt = TYPES[s["type"]]
    if s["kind"] == "dispatch":
        offsets, order, slot = _sorted_pairs(s["ids"], s["experts"])
        at = torch.arange(order.numel(), device=order.device)
        xs = torch.where((at < offsets[-1])[:, None], s["x"][order.long() // s["top_k"]], 0.0)
        out = {"offsets": offsets, "order": order, "slot": slot, "xs": xs.to(dt)}
        if s["grad"]:
            out["dx"] = _rows_of_pairs(s["dxs"], slot, slot < offsets[-1]).sum(1).to(dt)
        return out
    if s["kind"] == "combine":
        kept = s["slot"] < s["offsets"][-1]
        rows = _rows_of_pairs(s["h"], s["slot"], kept)
        out = {"y": (rows * s["weights"][..., None]).sum(1).to(dt)}
        if s["grad"]:
            dy = s["dy"].float()
            dh = torch.where(kept[..., None], s["weights"][..., None] * dy[:, None], 0.0)
            out["dh"] = dh.reshape(s["h"].shape).to(dt)[s["order"].long()]
            out["dw"] = (rows * dy[:, None]).sum(-1)
        return out
    if s["kind"] == "gemm":
        off, most, S = s["offsets"], s["most"], s["rows"]
        b = s["b"].float()
        if not s["grad"]:
            c = torch.bmm(_padded(s["a"], off, most), b.transpose(1, 2) if s["trans"] else b)
            return {"c": _unpadded(c, off, S).to(dt)}
        a, dc = _padded(s["a"], off, most), _padded(s["dc"], off, most)
        da = torch.bmm(dc, b if s["trans"] else b.transpose(1, 2))
        left, right = (dc, a) if s["trans"] else (a, dc)
        return {"da": _unpadded(da, off, S).to(dt), "db": torch.bmm(left.transpose(1, 2), right).to(dt)}
    q, scales, zeros = s["q"], s["scales"], s["zeros"]
    if s["ids"] is not None:
        at = s["ids"].long()
        q, scales = q[at], scales[at]
        zeros = zeros[at] if zeros is not None else None
    w = _nibbles(q).float().unflatten(-1, (-1, s["group"]))
    w = (w - (8.0 if zeros is None else zeros.float()[..., None])) * scales.float()[..., None]
    w = w.flatten(-2)
    x = s["x"].float()
    y = torch.bmm(w, x[:, :, None])[..., 0] if s["ids"] is not None else x @ w[0].t()
    return {"y": y.to(dt)}


def work(case):
    b = BYTES[case["type"]]
    if case["kind"] in ("dispatch", "combine"):
        T, P, d = case["tokens"], case["tokens"] * case["top_k"], case["width"]
        if case["kind"] == "dispatch":
            size = P * (8 if case["ids"] == "int64" else 4) + 8 * P + 4 * (case["experts"] + 1) + (T + P) * d * b
            return {"bytes": size + ((T + P) * d * b if case["grad"] else 0), "flops": P * d if case["grad"] else 0}
        # The gradients share the rows h with the forward pass: read once.
        size = (T + P) * d * b + 8 * P
        return {"bytes": size + ((T + P) * d * b + 4 * P if case["grad"] else 0),
                "flops": (5 if case["grad"] else 2) * P * d}
    K, N = case["k"], case["n"]
    if case["kind"] == "gemm":
        S = case["rows"]
        m = min(case["experts"], S) * K * N
        if case["grad"]:
            return {"bytes": (2 * S * K + S * N + m + case["experts"] * K * N) * b, "flops": 4 * S * K * N}
        return {"bytes": (S * K + S * N + m) * b, "flops": 2 * S * K * N}
    R, used = case["rows"], min(case["experts"], case["rows"])
    return {"bytes": used * N * (K // 2 + K // case["group"] * (b + (1 if case["zeros"] else 0))) + R * (K + N) * b,
            "flops": 2 * R * N * K}


def exact(case, seed):
    """The same outputs in 64 bits, from the definitions, one expert or choice at a time."""
    s = prepare(case, seed)
    if case["kind"] in ("dispatch", "combine"):
        T, k, E = case["tokens"], case["top_k"], case["experts"]
        if case["kind"] == "dispatch":
            flat = s["ids"].reshape(-1)
            parts = [torch.nonzero(flat == e)[:, 0] for e in range(E)]
            kept_pairs = torch.cat(parts)
            out = {"offsets": None, "order": None, "slot": None}
            xs = torch.zeros((T * k, case["width"]), dtype=torch.float64, device="cuda")
            xs[:kept_pairs.numel()] = s["x"].double()[kept_pairs // k]
            out["xs"] = xs
            if case["grad"]:
                dx = torch.zeros((T, case["width"]), dtype=torch.float64, device="cuda")
                out["dx"] = dx.index_add_(0, kept_pairs // k, s["dxs"][:kept_pairs.numel()].double())
            return out
        end = int(s["offsets"][-1])
        y = torch.zeros((T, case["width"]), dtype=torch.float64, device="cuda")
        dh = torch.zeros((T * k, case["width"]), dtype=torch.float64, device="cuda") if case["grad"] else None
        dw = torch.zeros((T, k), dtype=torch.float64, device="cuda")
        for j in range(k):
            t = torch.nonzero(s["slot"][:, j] < end)[:, 0]
            at = s["slot"][t, j].long()
            h, w = s["h"][at].double(), s["weights"][t, j].double()[:, None]
            y[t] += w * h
            if case["grad"]:
                dy = s["dy"][t].double()
                dh[at] = w * dy
                dw[t, j] = (dy * h).sum(1)
        return {"y": y, "dh": dh, "dw": dw} if case["grad"] else {"y": y}
    if case["kind"] == "gemm":
        off = s["offsets"].tolist()
        S, K, N, E = case["rows"], case["k"], case["n"], case["experts"]
        if not case["grad"]:
            c = torch.zeros((S, N), dtype=torch.float64, device="cuda")
            for e in range(E):
                w = s["b"][e].double()
                c[off[e]:off[e + 1]] = s["a"][off[e]:off[e + 1]].double() @ (w.t() if case["trans"] else w)
            return {"c": c}
        da = torch.zeros((S, K), dtype=torch.float64, device="cuda")
        db = torch.zeros(tuple(s["b"].shape), dtype=torch.float64, device="cuda")
        for e in range(E):
            a, dc, w = s["a"][off[e]:off[e + 1]].double(), s["dc"][off[e]:off[e + 1]].double(), s["b"][e].double()
            da[off[e]:off[e + 1]] = dc @ (w if case["trans"] else w.t())
            db[e] = dc.t() @ a if case["trans"] else a.t() @ dc
        return {"da": da, "db": db}
    y = torch.zeros((case["rows"], case["n"]), dtype=torch.float64, device="cuda")
    ids = [0] * case["rows"] if s["ids"] is None else s["ids"].tolist()
    G = case["group"]
    for e in sorted(set(ids)):
        rows = [r for r in range(case["rows"]) if ids[r] == e]
        x = s["x"][rows].double()
        for lo in range(0, case["k"], G):
            w = s["q"][e, :, lo // 2:(lo + G) // 2]
            z = s["zeros"][e, :, lo // G].double()[:, None] if case["zeros"] else 8.0
            part = x[:, lo:lo + G:2] @ ((w % 16).double() - z).t() + x[:, lo + 1:lo + G:2] @ ((w // 16).double() - z).t()
            y[rows] += part * s["scales"][e, :, lo // G].double()
    return {"y": y}

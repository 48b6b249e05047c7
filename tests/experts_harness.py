"""Helpers of the mixture-of-experts tests: 64-bit definitions written out on the CPU, strided device tensors, and
error bounds.

Bounds are derived, not tuned. A sum of n products held in fp32, each addition off by at most one unit in its last
place (2^-23, rounded or cut), is off by at most (n + 1) * 2^-23 * sum |terms|; ``bound`` allows twice that. Rounding to
the output type adds at most 2^-24 (fp32), 2^-8 (bf16) or 2^-11 (fp16) of the value; allowed are ROUNDING's."""

import numpy as np
import torch

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
ROUNDING = {torch.float32: 2.0 ** -23, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -10}
TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}
CANARY = 77.25


def bound(exact, magnitude, terms, dtype):
    return 2 * (terms + 1) * 2.0 ** -23 * magnitude + ROUNDING[dtype] * np.abs(exact) + TINY[dtype]


def assert_within(got, exact, limit, what=""):
    got = got.detach().double().cpu().numpy()
    assert got.shape == exact.shape, what
    off = np.abs(got - exact)
    bad = ~(off <= limit)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} out of bound, worst {np.nanmax(off / limit):.3g} of it"


def strided(t, pad=0, offset=0):
    """A CUDA copy of the 2-D tensor t with rows `pad` elements longer apart, `offset` elements into its buffer."""
    rows, cols = t.shape
    flat = torch.full((offset + max(rows, 1) * (cols + pad) + 16,), CANARY, dtype=t.dtype, device="cuda")
    view = flat.as_strided((rows, cols), (cols + pad, 1), offset)
    view.copy_(t)
    return view


def canaries_intact(view):
    """Whether everything around a strided() view is as it was."""
    flat = view.as_strided((view.untyped_storage().nbytes() // view.element_size(),), (1,), 0).clone()
    rows, cols = view.shape
    flat.as_strided((rows, cols), view.stride(), view.storage_offset()).fill_(CANARY)
    return bool((flat == CANARY).all())


def route64(ids, experts):
    """offsets, order and slot of sorted pairs, pair by pair."""
    flat = ids.reshape(-1).tolist()
    groups = [[] for _ in range(experts + 1)]
    for p, e in enumerate(flat):
        groups[e if 0 <= e < experts else experts].append(p)
    offsets = [0]
    for g in groups[:experts]:
        offsets.append(offsets[-1] + len(g))
    order = [p for g in groups for p in g]
    slot = [0] * len(flat)
    for s, p in enumerate(order):
        slot[p] = s
    return (np.array(offsets, np.int32), np.array(order, np.int32).reshape(-1),
            np.array(slot, np.int32).reshape(tuple(ids.shape)))


def random_ids(rng, tokens, top_k, experts, drop=0.0, skew=0.0):
    p = np.exp(skew * rng.standard_normal(experts))
    ids = rng.choice(experts, size=(tokens, top_k), p=p / p.sum())
    ids = np.where(rng.random((tokens, top_k)) < drop, rng.choice([-1, experts, experts + 7], size=(tokens, top_k)), ids)
    return torch.from_numpy(ids)


def offsets_of(counts):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32)

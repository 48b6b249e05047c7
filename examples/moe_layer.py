"""A mixture-of-experts layer on the library's operators: one training step, then single tokens from 4-bit experts.

The layer maps each token through its top_k experts, h = silu(x W1[e]) W2[e], and adds the results up with the
router's weights. ``forward`` and ``backward`` are the calls a training step makes; ``quantize`` and ``decode`` those
of a server. Run as a program it compares both with plain PyTorch and prints the errors::

    python examples/moe_layer.py [--tokens 512] [--experts 8] [--top-k 2] [--width 256] [--hidden 512] [--type bf16]
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from dense_fp32_matrix_major_gb300 import experts  # noqa: E402

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def forward(x, ids, weights, w1, w2):
    """The layer's output and what its backward pass needs. w1: experts x width x hidden, w2: experts x hidden x width."""
    r = experts.sort(ids, w1.shape[0])
    xs = experts.gather(x, r)
    pre = experts.gemm(xs, w1, r.offsets)
    act = torch.nn.functional.silu(pre)
    h = experts.gemm(act, w2, r.offsets)
    return experts.combine(h, weights, r), (r, xs, pre, act, h)


def backward(dy, weights, w1, w2, saved):
    """Gradients of x, the router's weights, w1 and w2."""
    r, xs, pre, act, h = saved
    dh, dweights = experts.combine_grad(dy, h, weights, r)
    dact = experts.gemm(dh, w2, r.offsets, transB=True)
    dw2 = experts.gemm_wgrad(act, dh, r.offsets)
    s = torch.sigmoid(pre.float())
    dpre = (dact.float() * (s * (1 + pre.float() * (1 - s)))).to(pre.dtype)
    dxs = experts.gemm(dpre, w1, r.offsets, transB=True)
    dw1 = experts.gemm_wgrad(xs, dpre, r.offsets)
    return experts.gather_grad(dxs, r), dweights, dw1, dw2


def quantize(w, group):
    """4-bit values, scales and zero points of experts x in x out matrices, as experts.w4_matvec takes them."""
    rows = w.transpose(1, 2).float().unflatten(-1, (-1, group))  # experts x out x groups x group
    low, high = rows.amin(-1), rows.amax(-1)
    scale = ((high - low) / 15).clamp(min=1e-8)
    zero = (-low / scale).round().clamp(0, 15)
    q = (rows / scale[..., None] + zero[..., None]).round().clamp(0, 15).to(torch.uint8).flatten(-2)
    return (q[..., 0::2] | (q[..., 1::2] << 4)).contiguous(), scale, zero.to(torch.uint8)


def dequantize(packed, group):
    """The experts x in x out matrices that the 4-bit values stand for."""
    q, scale, zero = packed
    v = torch.stack([q & 15, q >> 4], -1).flatten(-2).float().unflatten(-1, (-1, group))
    return ((v - zero.float()[..., None]) * scale[..., None]).flatten(-2).transpose(1, 2)


def decode(x, ids, weights, q1, q2, group):
    """The layer for a few tokens from 4-bit matrices: every (token, choice) pair is a row with its own expert."""
    top_k = ids.shape[1]
    pairs = ids.reshape(-1).to(torch.int32)
    pre = experts.w4_matvec(x.repeat_interleave(top_k, 0), *q1[:2], zeros=q1[2], group=group, ids=pairs)
    h = experts.w4_matvec(torch.nn.functional.silu(pre), *q2[:2], zeros=q2[2], group=group, ids=pairs)
    slot = torch.arange(pairs.numel(), dtype=torch.int32, device=x.device)
    offsets = torch.full((2,), pairs.numel(), dtype=torch.int32, device=x.device)  # pairs in their own order
    return experts.combine(h, weights, experts.Routing(offsets, slot, slot.reshape(ids.shape)))


def reference(x, ids, weights, w1, w2):
    """The layer in plain PyTorch and 64 bits."""
    y = torch.zeros_like(x)
    for e in range(w1.shape[0]):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        y = y.index_add(0, t, (torch.nn.functional.silu(x[t] @ w1[e]) @ w2[e]) * weights[t, j, None])
    return y


def error(got, want):
    return float((got.double() - want).norm() / want.norm())


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("tokens", 512), ("experts", 8), ("top-k", 2), ("width", 256), ("hidden", 512), ("group", 64)):
        ap.add_argument("--" + name, type=int, default=value)
    ap.add_argument("--type", choices=sorted(TYPES), default="bf16")
    a = ap.parse_args(argv)
    dt = TYPES[a.type]
    g = torch.Generator(device="cuda").manual_seed(1)

    def randn(*shape, scale=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(dt)

    x, dy = randn(a.tokens, a.width), randn(a.tokens, a.width)
    w1 = randn(a.experts, a.width, a.hidden, scale=a.width ** -0.5)
    w2 = randn(a.experts, a.hidden, a.width, scale=a.hidden ** -0.5)
    scores, ids = torch.randn((a.tokens, a.experts), generator=g, device="cuda").topk(a.top_k, dim=1)
    weights = torch.softmax(scores, 1)

    y, saved = forward(x, ids, weights, w1, w2)
    grads = backward(dy, weights, w1, w2, saved)
    leaves = [t.double().requires_grad_() for t in (x, weights, w1, w2)]
    want = reference(leaves[0], ids, *leaves[1:])
    want_grads = torch.autograd.grad(want, leaves, dy.double())
    errors = {"y": error(y, want.detach())}
    errors.update({n: error(got, w) for n, got, w in zip(("dx", "dweights", "dw1", "dw2"), grads, want_grads)})

    few = min(4, a.tokens)
    q1, q2 = quantize(w1, a.group), quantize(w2, a.group)
    tokens = decode(x[:few], ids[:few], weights[:few], q1, q2, a.group)
    want = reference(x[:few].double(), ids[:few], weights[:few].double(), dequantize(q1, a.group).double(),
                     dequantize(q2, a.group).double())
    errors["decode"] = error(tokens, want)
    for name, e in errors.items():
        print(f"{name:9s} relative error {e:.2e}")
    return errors


if __name__ == "__main__":
    main()

"""A mixture-of-experts layer trained in 8-bit floating point, then serving tokens from its 8-bit experts.

The layer maps each token through its top_k experts, h = W2[e] silu(W1[e] x), and adds the results up with the router's
weights. Every product reads e4m3 operands with a scale for each block of 128, gradients in e5m2 (:class:`ExpertLinear`);
master weights and their gradients stay in fp32. ``decode`` is the call of a server. Run as a program it compares both
with plain PyTorch in 64 bits and prints the errors, which are those of the 8-bit values::

    python examples/fp8_layer.py [--tokens 512] [--experts 8] [--top-k 2] [--width 256] [--hidden 512]
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from dense_fp32_matrix_major_gb300 import experts, fp8, layer  # noqa: E402


class ExpertLinear(torch.autograd.Function):
    """out[s] = x[s] W[e]^T for the rows s of group e, in 8-bit floating point."""

    @staticmethod
    def forward(ctx, x, w, offsets):
        w8 = fp8.quantize(w, "blocks")
        ctx.save_for_backward(x, offsets, *w8)
        return fp8.gemm(fp8.quantize(x, "rows"), w8, offsets, transB=True, dtype=x.dtype)

    @staticmethod
    def backward(ctx, dy):
        x, offsets, *w8 = ctx.saved_tensors
        dy = dy.contiguous()
        e5m2 = torch.float8_e5m2
        dx = fp8.gemm(fp8.quantize(dy, "rows", dtype=e5m2), fp8.Quantized(*w8), offsets, dtype=x.dtype)
        dw = fp8.gemm_wgrad(fp8.quantize(dy, "columns", dtype=e5m2, offsets=offsets),
                            fp8.quantize(x, "columns", offsets=offsets), offsets)
        return dx, dw, None


class Gather(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, routing):
        ctx.routing = routing
        return experts.gather(x, routing)

    @staticmethod
    def backward(ctx, dxs):
        return experts.gather_grad(dxs.contiguous(), ctx.routing), None


class Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, h, weights, routing):
        ctx.routing = routing
        ctx.save_for_backward(h, weights)
        return experts.combine(h, weights, routing)

    @staticmethod
    def backward(ctx, dy):
        dh, dweights = experts.combine_grad(dy.contiguous(), *ctx.saved_tensors, ctx.routing)
        return dh, dweights, None


def forward(x, ids, weights, w1, w2):
    """The layer of a training step. w1: experts x hidden x width, w2: experts x width x hidden, both fp32."""
    r = experts.sort(ids, w1.shape[0])
    h = torch.nn.functional.silu(ExpertLinear.apply(Gather.apply(x, r), w1, r.offsets))
    return Combine.apply(ExpertLinear.apply(h, w2, r.offsets), weights, r)


def decode(x, ids, weights, w1, w2):
    """The layer for a few tokens, w1 and w2 quantised once."""
    return layer.forward(x, ids, weights, w1, w2, activation="silu")


def reference(x, ids, weights, w1, w2):
    """The layer in plain PyTorch and 64 bits."""
    y = torch.zeros_like(x)
    for e in range(w1.shape[0]):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        y = y.index_add(0, t, (torch.nn.functional.silu(x[t] @ w1[e].t()) @ w2[e].t()) * weights[t, j, None])
    return y


def error(got, want):
    return float((got.double() - want).norm() / want.norm())


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("tokens", 512), ("experts", 8), ("top-k", 2), ("width", 256), ("hidden", 512)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args(argv)
    g = torch.Generator(device="cuda").manual_seed(1)

    def randn(*shape, scale=1.0):
        return torch.randn(shape, generator=g, device="cuda") * scale

    x, dy = randn(a.tokens, a.width).bfloat16(), randn(a.tokens, a.width).bfloat16()
    w1, w2 = randn(a.experts, a.hidden, a.width, scale=a.width ** -0.5), randn(a.experts, a.width, a.hidden,
                                                                               scale=a.hidden ** -0.5)
    scores, ids = randn(a.tokens, a.experts).topk(a.top_k, dim=1)
    weights = torch.softmax(scores, 1)

    leaves = [t.detach().requires_grad_() for t in (x, weights, w1, w2)]
    y = forward(leaves[0], ids, *leaves[1:])
    grads = torch.autograd.grad(y, leaves, dy)
    exact = [t.detach().double().requires_grad_() for t in (x, weights, w1, w2)]
    want = reference(exact[0], ids, *exact[1:])
    want_grads = torch.autograd.grad(want, exact, dy.double())
    errors = {"y": error(y.detach(), want.detach())}
    errors.update({n: error(got, w) for n, got, w in zip(("dx", "dweights", "dw1", "dw2"), grads, want_grads)})

    few = min(4, a.tokens)
    tokens = decode(x[:few], ids[:few], weights[:few], fp8.quantize(w1, "blocks"), fp8.quantize(w2, "blocks"))
    errors["decode"] = error(tokens, want[:few].detach())
    for name, e in errors.items():
        print(f"{name:9s} relative error {e:.2e}")
    return errors


if __name__ == "__main__":
    main()

"""The example layer: the operators together, forward, backward and from 4-bit matrices, against 64-bit autograd."""

import pytest
import torch

pytestmark = pytest.mark.gpu

# Of each type's rounding (2^-24, 2^-9, 2^-12 of a value, root mean square), up to five roundings in a row and
# the products' own error; the 4-bit layer is compared with what its matrices stand for.
LIMIT = {"f32": 1e-5, "bf16": 2e-2, "f16": 3e-3}


@pytest.mark.parametrize("kind", sorted(LIMIT))
@pytest.mark.parametrize("sizes", [(512, 8, 2, 256, 512), (33, 5, 3, 136, 200), (1, 4, 4, 64, 64)])
def test_layer(kind, sizes):
    from examples import moe_layer

    tokens, experts, top_k, width, hidden = sizes
    group = 32 if width % 64 or hidden % 64 else 64
    width, hidden = (width + group - 1) // group * group, (hidden + group - 1) // group * group
    errors = moe_layer.main(["--tokens", str(tokens), "--experts", str(experts), "--top-k", str(top_k), "--width",
                             str(width), "--hidden", str(hidden), "--group", str(group), "--type", kind])
    assert set(errors) == {"y", "dx", "dweights", "dw1", "dw2", "decode"}
    for name, e in errors.items():
        assert e <= LIMIT[kind], (name, e)


def test_offsets_past_32_bits():
    """Element offsets beyond 2^31: rows, products per expert and 4-bit matrices; spot checks at both ends."""
    from dense_fp32_matrix_major_gb300 import experts

    tokens, top_k, E, width = 300000, 4, 4, 2048
    ids = (torch.arange(tokens * top_k, device="cuda").reshape(tokens, top_k) * 7 // 3 % E).to(torch.int32)
    r = experts.sort(ids, E)
    x = torch.randn(tokens, width, device="cuda", dtype=torch.bfloat16)
    xs = experts.gather(x, r)
    assert xs.numel() > 2 ** 31
    for s in (0, 12345, tokens * top_k // 2, tokens * top_k - 1):
        assert torch.equal(xs[s], x[r.order[s].item() // top_k])
    dx = experts.gather_grad(xs, r)
    assert torch.equal(dx, x * top_k)
    dh, dw = experts.combine_grad(x, xs, torch.full((tokens, top_k), 0.5, device="cuda"), r)
    for s in (0, tokens * top_k - 1):
        assert torch.equal(dh[s], xs[s] * 0.5)
    want = (x.float() * x.float()).sum(1)
    assert torch.allclose(dw, want[:, None].expand(-1, top_k), rtol=1e-5)
    del dh, dx
    b = torch.randn(E, width, 128, device="cuda", dtype=torch.bfloat16)
    c = experts.gemm(xs, b, r.offsets)
    for s in (0, tokens * top_k // 2, tokens * top_k - 1):
        e = ids.reshape(-1)[r.order[s]].item()
        want = xs[s].double() @ b[e].double()
        assert float((c[s].double() - want).norm() / want.norm()) < 4e-3
    db = experts.gemm_wgrad(xs, c, r.offsets)
    o = r.offsets.tolist()
    want = xs[o[E - 1]:o[E]].float().t() @ c[o[E - 1]:o[E]].float()
    assert float((db[E - 1].float() - want).norm() / want.norm()) < 4e-3
    del xs, c
    E, N, K = 40, 16384, 8192
    q = torch.randint(0, 256, (E, N, K // 2), device="cuda", dtype=torch.uint8)
    assert q.numel() > 2 ** 31
    scales = torch.ones(E, N, K // 128, device="cuda", dtype=torch.bfloat16)
    xr = torch.randn(2, K, device="cuda")
    pick = torch.tensor([0, E - 1], dtype=torch.int32, device="cuda")
    y = experts.w4_matvec(xr, q, scales, group=128, ids=pick)
    for i, e in enumerate(pick.tolist()):
        w = torch.stack([q[e] & 15, q[e] >> 4], -1).flatten(-2).double() - 8
        want = w @ xr[i].double()
        assert float((y[i].double() - want).norm() / want.norm()) < 1e-5

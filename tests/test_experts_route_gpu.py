"""Sort by expert, gather, combine and their gradients against 64-bit definitions."""

import numpy as np
import pytest
import torch

from tests.experts_harness import (DTYPES, assert_within, bound, canaries_intact, random_ids, route64, strided)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ex():
    from dense_fp32_matrix_major_gb300 import experts

    return experts


SORT = [
    # tokens, top_k, experts, dropped share, skew
    (0, 2, 8, 0.0, 0.0), (1, 1, 1, 0.0, 0.0), (1, 1, 4, 1.0, 0.0), (5, 3, 7, 0.3, 0.0), (33, 2, 8, 0.0, 2.0),
    (64, 1, 256, 0.1, 0.0), (1000, 8, 60, 0.05, 1.0), (4097, 2, 33, 0.0, 3.0), (1, 64, 4096, 0.2, 0.0),
    (12289, 1, 2, 0.5, 0.0), (10007, 6, 160, 0.02, 1.0), (3000, 5, 4096, 0.1, 0.0), (66000, 8, 256, 0.01, 1.0),
    (20011, 1, 1, 0.0, 0.0),
]


@pytest.mark.parametrize("tokens,top_k,experts,drop,skew", SORT)
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_sort(ex, tokens, top_k, experts, drop, skew, dtype):
    ids = random_ids(np.random.default_rng(tokens + experts), tokens, top_k, experts, drop, skew).to(dtype)
    offsets, order, slot = route64(ids, experts)
    for _ in range(2):
        r = ex.sort(ids.cuda(), experts)
        assert r.offsets.dtype == r.order.dtype == r.slot.dtype == torch.int32
        assert np.array_equal(r.offsets.cpu().numpy(), offsets)
        assert np.array_equal(r.order.cpu().numpy(), order)
        assert np.array_equal(r.slot.cpu().numpy(), slot)


def test_sort_takes_ids_beyond_32_bits_as_dropped(ex):
    ids = torch.tensor([[1, 1 << 32], [-(1 << 40), 0]], dtype=torch.int64, device="cuda")
    r = ex.sort(ids, 2)
    assert r.offsets.tolist() == [0, 1, 2]
    assert r.order.tolist() == [3, 0, 1, 2]


ROWS = [
    # tokens, top_k, experts, width, row padding, buffer offset, dropped share
    (1, 1, 1, 1, 0, 0, 0.0), (1, 4, 8, 1024, 0, 0, 0.0), (3, 2, 4, 33, 0, 0, 0.4), (7, 9, 16, 130, 2, 2, 0.2),
    (64, 2, 8, 256, 8, 0, 0.0), (65, 3, 5, 1537, 0, 0, 0.1), (33, 17, 64, 100, 4, 4, 0.3), (500, 8, 60, 2048, 0, 0, 0.05),
    (40, 2, 4, 4100, 0, 1, 0.5), (9, 2, 4, 64, 0, 0, 1.0),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("tokens,top_k,experts,width,pad,offset,drop", ROWS)
def test_rows(ex, dtype, tokens, top_k, experts, width, pad, offset, drop):
    """gather, its gradient, combine and its gradients, with NaN in every row that must not be read."""
    dt = DTYPES[dtype]
    rng = np.random.default_rng(tokens * 31 + width)
    ids = random_ids(rng, tokens, top_k, experts, drop).to(torch.int32)
    offsets, order, slot = route64(ids, experts)
    pairs, end = tokens * top_k, offsets[-1]
    r = ex.sort(ids.cuda(), experts)

    def values(rows):
        return torch.from_numpy(rng.standard_normal((rows, width)).astype(np.float32)).to(dt)

    x, h, dy = values(tokens), values(pairs), values(tokens)
    w = torch.from_numpy(rng.random((tokens, top_k)).astype(np.float32))
    kept = slot < end
    h[end:] = float("nan")
    w[torch.from_numpy(~kept)] = float("nan")
    x64, h64, dy64, w64 = x.double().numpy(), h.double().numpy(), dy.double().numpy(), w.double().numpy()
    rows64 = np.where(kept[..., None], h64[slot], 0.0)
    wk = np.where(kept, w64, 0.0)

    out = strided(torch.zeros(pairs, width, dtype=dt), pad, offset)
    xs = ex.gather(strided(x, pad, offset), r, out=out)
    want = np.zeros((pairs, width))
    want[slot[kept]] = np.broadcast_to(x64[:, None], rows64.shape)[kept]
    assert np.array_equal(xs.double().cpu().numpy(), want)
    assert canaries_intact(out)

    dx = ex.gather_grad(strided(h, pad, offset), r)
    assert_within(dx, rows64.sum(1), bound(rows64.sum(1), np.abs(rows64).sum(1), top_k, dt), "dx")

    out = strided(torch.zeros(tokens, width, dtype=dt), pad, offset)
    y = ex.combine(strided(h, pad, offset), w.cuda(), r, out=out)
    terms = rows64 * wk[..., None]
    assert_within(y, terms.sum(1), bound(terms.sum(1), np.abs(terms).sum(1), top_k, dt), "y")
    assert canaries_intact(out)

    dh, dw = ex.combine_grad(strided(dy, pad, offset), strided(h, pad, offset), w.cuda(), r)
    want = np.zeros((pairs, width))
    want[slot[kept]] = (wk[..., None] * dy64[:, None])[kept]
    assert_within(dh, want, bound(want, np.abs(want), 1, dt), "dh")
    prod = rows64 * dy64[:, None]
    assert dw.dtype == torch.float32
    assert_within(dw, prod.sum(-1), bound(prod.sum(-1), np.abs(prod).sum(-1), width, torch.float32), "dw")


def test_gradients_against_differences(ex):
    """combine is linear in h and in w, gather in x: differences over a step of one equal the gradients."""
    rng = np.random.default_rng(5)
    tokens, top_k, experts, width = 37, 3, 6, 70
    ids = random_ids(rng, tokens, top_k, experts, 0.2).to(torch.int32)
    r = ex.sort(ids.cuda(), experts)

    def cuda(*shape):
        return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).cuda()

    h, u, w, v = cuda(tokens * top_k, width), cuda(tokens * top_k, width), cuda(tokens, top_k), cuda(tokens, top_k)
    dy, x, dxs = cuda(tokens, width), cuda(tokens, width), cuda(tokens * top_k, width)

    def dot(a, b):
        return float((a.double() * b.double()).sum())

    dh, dw = ex.combine_grad(dy, h, w, r)
    # Each value carries a few fp32 roundings of its own size; their sum over all is far below this.
    tol = 1e-5 * tokens * top_k * width
    along_h = (dot(dy, ex.combine(h + u, w, r)) - dot(dy, ex.combine(h - u, w, r))) / 2
    along_w = (dot(dy, ex.combine(h, w + v, r)) - dot(dy, ex.combine(h, w - v, r))) / 2
    assert abs(along_h - dot(dh, u)) <= tol
    assert abs(along_w - dot(dw, v)) <= tol
    y = cuda(tokens, width)
    along_x = (dot(dxs, ex.gather(x + y, r)) - dot(dxs, ex.gather(x - y, r))) / 2
    assert abs(along_x - dot(ex.gather_grad(dxs, r), y)) <= tol


def test_non_finite_rows_stay_in_their_token(ex):
    ids = torch.tensor([[0, 1], [1, 0], [0, -1]], dtype=torch.int32, device="cuda")
    r = ex.sort(ids, 2)
    h = torch.ones(6, 8, device="cuda")
    h[r.slot[1, 0].item()] = float("inf")
    w = torch.full((3, 2), 0.5, device="cuda")
    y = ex.combine(h, w, r).cpu()
    assert (y[0] == 1).all() and torch.isinf(y[1]).all() and (y[2] == 0.5).all()
    w[1, 0] = 0.0
    assert torch.isnan(ex.combine(h, w, r)[1]).all()  # 0 * inf


def test_slots_and_offsets_out_of_range_touch_nothing(ex):
    """Bad slots count as dropped; bad offsets are limited to the pairs."""
    slot = torch.tensor([[0, 99], [-5, 3]], dtype=torch.int32, device="cuda")
    r = ex.Routing(torch.tensor([0, 2, 1 << 30], dtype=torch.int32, device="cuda"),
                   torch.arange(4, dtype=torch.int32, device="cuda"), slot)
    x = torch.arange(1, 17, dtype=torch.float32, device="cuda").reshape(2, 8)
    out = strided(torch.zeros(4, 8), 0, 8)
    ex.gather(x, r, out=out)
    assert torch.equal(out[0], x[0]) and torch.equal(out[3], x[1]) and (out[1:3] == 0).all()
    assert canaries_intact(out)
    y = ex.combine(out, torch.ones(2, 2, device="cuda"), r)
    assert torch.equal(y, x)
    dh, dw = ex.combine_grad(x, out, torch.ones(2, 2, device="cuda"), r)
    assert torch.equal(dw[:, 0].cpu(), torch.tensor([float((x[0] * x[0]).sum()), 0.0]))
    assert torch.equal(dh[0], x[0]) and torch.equal(dh[3], x[1])


def test_other_stream(ex):
    """Inputs made on one stream, the calls on another that waits for it."""
    ids = torch.randint(0, 16, (3000, 4), device="cuda")
    x = torch.randn(3000, 512, device="cuda")
    r0 = ex.sort(ids, 16)
    want = ex.gather_grad(ex.gather(x, r0), r0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    r = ex.sort(ids, 16, stream=side)
    got = ex.gather_grad(ex.gather(x, r, stream=side), r, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want) and torch.equal(r.order, r0.order)


def test_refusals(ex):
    ids = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    r = ex.sort(ids, 3)
    x = torch.zeros(4, 8, device="cuda")
    with pytest.raises(TypeError):
        ex.sort(ids.float(), 3)
    with pytest.raises(TypeError):
        ex.sort(ids.t(), 3)
    with pytest.raises(ex.SgemmError):
        ex.sort(ids, 5000)
    with pytest.raises(ValueError):
        ex.gather(x[:3], r)
    with pytest.raises(ValueError):
        ex.gather(torch.zeros(8, 4, device="cuda").t(), r)
    with pytest.raises(ValueError):
        ex.gather(x, r, out=torch.zeros(7, 8, device="cuda"))
    with pytest.raises(TypeError):
        ex.gather(x, r, out=torch.zeros(8, 8, dtype=torch.float16, device="cuda"))
    with pytest.raises(ex.SgemmError):
        buf = torch.zeros(12, 8, device="cuda")
        ex.gather(buf[:4], r, out=buf[2:10])  # overlaps its input
    with pytest.raises(TypeError):
        ex.combine(torch.zeros(8, 8, device="cuda"), torch.zeros(4, 2, dtype=torch.float16, device="cuda"), r)
    with pytest.raises(ValueError):
        ex.combine(torch.zeros(8, 8, device="cuda"), torch.zeros(2, 4, device="cuda"), r)

"""4-bit products at the sizes where their kernels change form: x at the limits of what stays in shared memory, streamed
x in several launches, rows without an expert."""

import numpy as np
import pytest
import torch

from tests.experts_harness import DTYPES, assert_within, bound

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ex():
    from dense_fp32_matrix_major_gb300 import experts

    return experts


def case(dtype, rows, N, K, group, experts=1, seed=0):
    """x, q, scales, zero points on the GPU, and the experts' matrices in 64 bits."""
    g = torch.Generator(device="cuda").manual_seed(rows * 7919 + N + K + seed)
    x = torch.randn((rows, K), generator=g, device="cuda").to(DTYPES[dtype])
    q = torch.randint(0, 256, (experts, N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = torch.rand((experts, N, -(-K // group)), generator=g, device="cuda") + 0.5
    z = torch.randint(0, 16, scales.shape, generator=g, device="cuda", dtype=torch.uint8)
    v = torch.stack([q & 15, q >> 4], -1).flatten(-2).double()
    at = torch.arange(K, device="cuda") // group
    return x, q, scales, z, (v - z.double()[..., at]) * scales.double()[..., at]


def check(y, x, w, ids, K, group, dtype):
    rows, experts = x.shape[0], w.shape[0]
    want, mag = torch.zeros(y.shape, dtype=torch.float64), torch.zeros(y.shape, dtype=torch.float64)
    at = np.zeros(rows, int) if ids is None else ids.cpu().numpy()
    for e in range(experts):
        r = np.nonzero(at == e)[0]
        if r.size:
            want[r] = (x[r].double() @ w[e].t()).cpu()
            mag[r] = (x[r].double().abs() @ w[e].abs().t()).cpu()
    # Terms: each x is up to three, each group's sum is scaled once.
    assert_within(y, want.numpy(), bound(want.numpy(), mag.numpy(), 3 * K + K // group + 2, DTYPES[dtype]))


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("rows,N,K", [(3, 200, 4096), (4, 2100, 4096), (5, 4900, 4096), (4, 700, 8192), (5, 1000, 3040)])
def test_three_to_five_fp32_rows(ex, rows, N, K, group):
    x, q, s, z, w = case("f32", rows, N, K, group)
    check(ex.w4_matvec(x, q, s, group=group, zeros=z), x, w, None, K, group, "f32")


# The last K for which x stays in shared memory, and the first for which it is streamed (k in steps of 256).
LIMITS = [("f32", 2, 6144), ("f32", 5, 3040), ("f32", 8, 2048), ("bf16", 8, 6144), ("f16", 8, 6144),
          ("bf16", 1, 73728), ("f16", 1, 73728)]


@pytest.mark.parametrize("dtype,rows,K", LIMITS)
@pytest.mark.parametrize("past", [False, True])
def test_limits_of_x_in_shared_memory(ex, dtype, rows, K, past):
    K += 64 if past else 0
    group = 128 if dtype != "f16" else 64
    x, q, s, z, w = case(dtype, rows, 70, K, group)
    check(ex.w4_matvec(x, q, s, group=group, zeros=z), x, w, None, K, group, dtype)


@pytest.mark.parametrize("dtype,rows,K", [("bf16", 600, 8192), ("f32", 700, 4096)])
def test_streamed_x_with_ids_in_several_launches(ex, dtype, rows, K):
    """More passes than one launch takes, x streamed, some rows without an expert, twice in a row."""
    x, q, s, z, w = case(dtype, rows, 40, K, 128, experts=5)
    g = torch.Generator(device="cuda").manual_seed(rows)
    ids = torch.randint(-1, 6, (rows,), generator=g, device="cuda", dtype=torch.int32)
    first = ex.w4_matvec(x, q, s, group=128, zeros=z, ids=ids)
    second = ex.w4_matvec(x, q, s, group=128, zeros=z, ids=ids)
    check(first, x, w, ids, K, 128, dtype)
    assert torch.equal(first, second)
    assert (first[(ids < 0) | (ids > 4)] == 0).all()


@pytest.mark.parametrize("dtype", ["f16", "f32"])
def test_streamed_x_of_many_rows(ex, dtype):
    """256 passes of eight rows a launch, and a part of a pass after two of them."""
    rows, K = 2 * 256 * 8 + 3, 6272
    x, q, s, z, w = case(dtype, rows, 24, K, 128)
    y = ex.w4_matvec(x, q, s, group=128, zeros=z)
    check(y, x, w, None, K, 128, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_streamed_x_of_rows_without_an_expert(ex, dtype):
    """No pass has work: zeros, and what follows on the stream is not disturbed."""
    K, rows = 8192, 9
    x, q, s, z, w = case(dtype, rows, 200, K, 64, experts=3)
    none = torch.full((rows,), -1, dtype=torch.int32, device="cuda")
    some = torch.tensor([2, 0, 1, 1, -1, 2, 0, 7, 1], dtype=torch.int32, device="cuda")
    x[4] = x[7] = float("nan")  # rows without an expert
    for _ in range(5):
        y = torch.ones((rows, 200), dtype=x.dtype, device="cuda")
        ex.w4_matvec(x, q, s, group=64, zeros=z, ids=none, out=y)
        again = ex.w4_matvec(x, q, s, group=64, zeros=z, ids=some)
        assert (y == 0).all()
        check(again, torch.nan_to_num(x), w, some, K, 64, dtype)

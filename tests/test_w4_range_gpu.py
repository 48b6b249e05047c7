"""4-bit products of values far apart: a large x whose q is the zero point adds nothing, and nothing overflows on the
way to a result that fits."""

import numpy as np
import pytest
import torch

from tests.experts_harness import DTYPES, assert_within, bound

N, K, GROUP = 64, 512, 128


@pytest.fixture(scope="module")
def ex():
    from dense_fp32_matrix_major_gb300 import experts

    return experts


def outliers(dtype, zeros, seed):
    """q (N x K), zero points (N x groups), x (3 x K) with a value of 60000 in each group where q is the zero point, and
    a small one at every 16th k; the products in 64 bits, the sum of their magnitudes and their number."""
    rng = np.random.default_rng(seed)
    q = rng.integers(0, 16, (N, K))
    z = rng.integers(0, 16, (N, K // GROUP)) if zeros else np.full((N, K // GROUP), 8)
    x = np.zeros((3, K), np.float32)
    x[:, ::16] = rng.standard_normal((3, K // 16)) * 2.0 ** -8
    for g in range(K // GROUP):
        x[:, g * GROUP + 5] = 60000.0 * (-1) ** g
        q[:, g * GROUP + 5] = z[:, g]
    x = torch.from_numpy(x).to(DTYPES[dtype])
    x64, w = x.double().numpy(), (q - np.repeat(z, GROUP, 1)).astype(np.float64)
    return q, z, x, x64 @ w.T, np.abs(x64) @ np.abs(w).T, K // 16


def limit(want, mag, terms, dtype):
    # Products of the outliers are 0 and add no error; an fp32 x has three terms, each group's sum is scaled once.
    return bound(want, mag, 3 * terms + K // GROUP + 2, DTYPES[dtype])


@pytest.mark.parametrize("dtype,zeros,base", [("f16", False, 0), ("f16", True, 0), ("bf16", False, 0), ("bf16", True, 8)])
def test_limit_notices_zero_points_taken_from_sums(dtype, zeros, base):
    """sum (q - base) x - (zero - base) sum x in 32 bits, which the limit below must not let pass."""
    q, z, x, want, mag, terms = outliers(dtype, zeros, 3)
    x32, got = x.float().numpy(), np.zeros((3, N), np.float32)
    for g in range(K // GROUP):
        sums, total = np.zeros((3, N), np.float32), np.zeros((3, 1), np.float32)
        for k in range(g * GROUP, (g + 1) * GROUP):
            sums += x32[:, k:k + 1] * (q[:, k] - base).astype(np.float32)
            total += x32[:, k:k + 1]
        got += sums - (z[:, g] - base).astype(np.float32) * total
    assert (np.abs(got - want) > 4 * limit(want, mag, terms, dtype)).any()


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [1, 3])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_outliers_at_the_zero_point_leave_no_trace(ex, dtype, zeros, rows):
    q, z, x, want, mag, terms = outliers(dtype, zeros, 3)
    packed = torch.from_numpy((q[:, ::2] | (q[:, 1::2] << 4)).astype(np.uint8)).cuda()
    y = ex.w4_matvec(x[:rows].cuda(), packed, torch.ones(N, K // GROUP, device="cuda"), group=GROUP,
                     zeros=torch.from_numpy(z.astype(np.uint8)).cuda() if zeros else None)
    assert_within(y, want[:rows], limit(want, mag, terms, dtype)[:rows])


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [1, 2, 4, 8])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("zeros", [False, True])
def test_sums_that_overflow_before_their_scale(ex, dtype, zeros, rows):
    """Values near the type's largest, weights up to 15, scales that bring the result back; pairs that cancel."""
    rng = np.random.default_rng(rows)
    q = rng.integers(0, 16, (N, K))
    z = rng.integers(0, 16, (N, K // GROUP)) if zeros else np.full((N, K // GROUP), 8)
    scales = (2.0 ** -rng.integers(7, 12, (N, K // GROUP))).astype(np.float32)
    x = rng.standard_normal((rows, K)).astype(np.float32)
    x[:, 3], x[:, 70], x[:, 200] = 1.0e38, -3.0e38, 2.5e38
    x[:, 300], x[:, 301] = 3.0e38, -3.0e38
    q[: N // 2, 301] = q[: N // 2, 300]  # these leave the small values' sum
    q[: N // 4, [3, 70, 200]] = z[: N // 4, [0, 0, 1]]
    x = torch.from_numpy(x).to(DTYPES[dtype])
    w = (q - np.repeat(z, GROUP, 1)) * np.repeat(scales.astype(np.float64), GROUP, 1)
    x64 = x.double().numpy()
    want, mag = x64 @ w.T, np.abs(x64) @ np.abs(w).T
    assert (np.abs(want) < 1e36).any() and (np.abs(want) > 1e36).any() and np.abs(want).max() < 3e38
    packed = torch.from_numpy((q[:, ::2] | (q[:, 1::2] << 4)).astype(np.uint8)).cuda()
    y = ex.w4_matvec(x.cuda(), packed, torch.from_numpy(scales).cuda(), group=GROUP,
                     zeros=torch.from_numpy(z.astype(np.uint8)).cuda() if zeros else None)
    assert torch.isfinite(y).all()
    assert_within(y, want, bound(want, mag, 3 * K + K // GROUP + 2, DTYPES[dtype]))


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [1, 2, 4, 8])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_infinities_and_nan(ex, dtype, rows):
    """The kinds of results are those of 64-bit sums, in every form of the kernel."""
    rng = np.random.default_rng(9)
    q = rng.integers(0, 16, (N, K))
    x = rng.standard_normal((rows, K)).astype(np.float32)
    x[0, 17] = np.inf
    if rows > 1:
        x[1, 9], x[1, 400] = np.inf, -np.inf
    if rows > 2:
        x[2, 500] = np.nan
    with np.errstate(invalid="ignore"):
        w = (q - 8).astype(np.float64)
        want = np.stack([(r[None] * w).sum(1) for r in x.astype(np.float64)])
    packed = torch.from_numpy((q[:, ::2] | (q[:, 1::2] << 4)).astype(np.uint8)).cuda()
    y = ex.w4_matvec(torch.from_numpy(x).to(DTYPES[dtype]).cuda(), packed, torch.ones(N, K // GROUP, device="cuda"),
                     group=GROUP).double().cpu().numpy()
    assert np.array_equal(np.isnan(y), np.isnan(want))
    assert np.array_equal(np.isposinf(y), np.isposinf(want)) and np.array_equal(np.isneginf(y), np.isneginf(want))


@pytest.mark.gpu
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_time_of_rows_that_are_not_finite(ex, dtype, value):
    """Such rows are not summed again (9.8 ms here, 0.04 ms otherwise): the products are IEEE's as they are."""
    rows, n, k = 8, 16384, 8192
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randint(0, 256, (n, k // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = torch.rand((n, k // 128), generator=g, device="cuda")
    x = torch.randn((rows, k), generator=g, device="cuda").to(DTYPES[dtype])
    x[:, k - 1] = value
    y = torch.empty((rows, n), dtype=x.dtype, device="cuda")
    times = []
    for _ in range(4):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        ex.w4_matvec(x, q, scales, group=128, out=y)
        b.record()
        b.synchronize()
        times.append(a.elapsed_time(b))
    assert min(times) < 2.0
    last = (q[:, -1] >> 4).float() - 8
    if value != value:
        assert torch.isnan(y).all()
    else:
        assert torch.equal(torch.isnan(y), (last == 0).expand(rows, n))
        assert torch.equal(torch.sign(y.float()[:, last != 0]), torch.sign(last[last != 0]).expand(rows, -1))

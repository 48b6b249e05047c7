"""Matrix-vector products with 4-bit weights against 64-bit sums."""

import numpy as np
import pytest
import torch

from tests.experts_harness import DTYPES, assert_within, bound, canaries_intact, strided

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ex():
    from dense_fp32_matrix_major_gb300 import experts

    return experts


def _weights(rng, E, N, K, group, zeros):
    G = -(-K // group)
    q = rng.integers(0, 256, (E, N, K // 2), dtype=np.uint8)
    scales = rng.uniform(0.5, 1.5, (E, N, G)).astype(np.float32)
    z = rng.integers(0, 16, (E, N, G), dtype=np.uint8) if zeros else None
    return q, scales, z


def _dense(q, scales, z, group):
    """The matrices in 64 bits."""
    E, N, half = q.shape
    v = np.empty((E, N, 2 * half))
    v[..., 0::2], v[..., 1::2] = q & 15, q >> 4
    at = np.arange(2 * half) // group
    return (v - (8 if z is None else z.astype(np.float64)[..., at])) * scales.astype(np.float64)[..., at]


def _check(ex, rng, dt, rows, N, K, group, *, experts=1, ids=None, zeros=False, scale_dt=torch.float32, pad=0, offset=0):
    q, scales, z = _weights(rng, experts, N, K, group, zeros)
    scales = torch.from_numpy(scales).to(scale_dt)
    x = torch.from_numpy(rng.standard_normal((rows, K)).astype(np.float32)).to(dt)
    w = _dense(q, scales.double().numpy(), z, group)
    x64 = x.double().numpy()
    at = np.zeros(rows, int) if ids is None else np.asarray(ids)
    want, mag = np.zeros((rows, N)), np.zeros((rows, N))
    for r in range(rows):
        if 0 <= at[r] < experts:
            want[r], mag[r] = w[at[r]] @ x64[r], np.abs(w[at[r]]) @ np.abs(x64[r])
    out = strided(torch.zeros(rows, N, dtype=dt), pad, offset)
    y = ex.w4_matvec(strided(x, pad, offset), torch.from_numpy(q).cuda(), scales.cuda(), group=group,
                     zeros=None if z is None else torch.from_numpy(z).cuda(),
                     ids=None if ids is None else torch.tensor(ids, dtype=torch.int32, device="cuda"), out=out)
    # Terms: each x is up to three, each group's sum is scaled once.
    assert_within(y, want, bound(want, mag, 3 * K + K // group + 2, dt), f"{rows} x {N} x {K}")
    assert canaries_intact(out)


SHAPES = [
    # rows, N, K, group
    (1, 1, 2, 32), (1, 16, 128, 128), (1, 17, 128, 32), (2, 31, 64, 64), (3, 100, 96, 32), (1, 64, 4096, 128),
    (5, 129, 1024, 64), (8, 256, 2048, 256), (9, 48, 640, 128), (16, 33, 320, 64), (17, 300, 512, 128), (8, 1000, 8192, 128),
    (7, 65, 130, 64), (2, 40, 1538, 128), (1, 2500, 352, 32), (33, 16, 128, 128), (1, 20, 12288, 256),
]


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,N,K,group", SHAPES)
def test_dense(ex, dtype, rows, N, K, group, zeros):
    rng = np.random.default_rng(rows * 1000 + N + K)
    _check(ex, rng, DTYPES[dtype], rows, N, K, group, zeros=zeros)


@pytest.mark.parametrize("scales", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_scale_types_and_strides(ex, dtype, scales):
    rng = np.random.default_rng(8)
    _check(ex, rng, DTYPES[dtype], 4, 70, 256, 64, zeros=True, scale_dt=DTYPES[scales], pad=3, offset=1)


IDS = [
    [0], [-1], [2, 2, 2], [0, 3, 1, 2, 0, 3], [4, -1, 0, 99, 3], [1] * 20, [0, 1] * 13, [3] * 8 + [1] + [3] * 8 + [-7],
]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("ids", IDS, ids=[str(i) for i in range(len(IDS))])
def test_experts(ex, dtype, ids):
    rng = np.random.default_rng(len(ids))
    _check(ex, rng, DTYPES[dtype], len(ids), 90, 384, 128, experts=4, ids=ids, zeros=True)
    _check(ex, rng, DTYPES[dtype], len(ids), 33, 160, 32, experts=4, ids=ids)


def test_many_rows_of_one_expert(ex):
    rng = np.random.default_rng(1)
    _check(ex, rng, torch.bfloat16, 700, 32, 128, 64, experts=3, ids=rng.integers(0, 3, 700).tolist())


def test_rows_do_not_mix(ex):
    """NaN and infinities stay in their row, and the other rows keep their bits."""
    rng = np.random.default_rng(4)
    q, scales, _ = _weights(rng, 1, 64, 512, 128, False)
    q, scales = torch.from_numpy(q[0]).cuda(), torch.from_numpy(scales[0]).cuda()
    for dt in DTYPES.values():
        x = torch.from_numpy(rng.standard_normal((6, 512)).astype(np.float32)).to(dt).cuda()
        all_rows = ex.w4_matvec(x, q, scales, group=128)
        x[2, 7], x[4, 9] = float("nan"), float("inf")
        y = ex.w4_matvec(x, q, scales, group=128)
        keep = [0, 1, 3, 5]
        assert torch.equal(y[keep], all_rows[keep])
        assert torch.isnan(y[2]).all()
        value = ((q[:, 4] >> 4) & 15).float() - 8  # k = 9
        assert torch.equal(torch.isnan(y[4]), value == 0)
        assert torch.equal(torch.sign(y[4][value != 0].float()), torch.sign(value[value != 0]))


def test_large_and_small_fp32(ex):
    """The three terms of an fp32 value cover its range: near overflow and down to small numbers."""
    q = torch.full((16, 64), 0x99, dtype=torch.uint8, device="cuda")  # every weight 1
    scales = torch.ones(16, 1, device="cuda")
    for value in (3.0e38, 1.2345678e-20, 16777215.0, 1.0000001, -2.9999998):
        x = torch.zeros(1, 128, device="cuda")
        x[0, 77] = value
        assert torch.equal(ex.w4_matvec(x, q, scales, group=128)[0], x[0, 77].expand(16))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("zeros", [False, True])
def test_outliers(ex, dtype, zeros):
    """Values of x a thousand times the others where q is the zero point: they must leave no trace in the sum."""
    rng = np.random.default_rng(12)
    dt, N, K, group = DTYPES[dtype], 64, 1024, 128
    q, scales, z = _weights(rng, 1, N, K, group, zeros)
    v = np.empty((N, K), dtype=np.uint8)
    v[:, 0::2], v[:, 1::2] = q[0] & 15, q[0] >> 4
    x = rng.standard_normal((3, K)).astype(np.float32)
    for g in range(K // group):
        x[:, g * group + 5] = 1000.0 * (g + 1)
        v[:, g * group + 5] = 8 if z is None else z[0, :, g]
    q[0] = v[:, 0::2] | (v[:, 1::2] << 4)
    x = torch.from_numpy(x).to(dt)
    w = _dense(q, scales.astype(np.float64), z, group)[0]
    want, mag = x.double().numpy() @ w.T, np.abs(x.double().numpy()) @ np.abs(w).T
    y = ex.w4_matvec(x.cuda(), torch.from_numpy(q[0]).cuda(), torch.from_numpy(scales[0]).cuda(), group=group,
                     zeros=None if z is None else torch.from_numpy(z[0]).cuda())
    # Zero points are taken from sums of q (fp16) or q - 8 (bf16): the outlier's share of those, at most 15 of it,
    # is cut at each of a group's 8 matrix instructions and rounded twice when it is taken out (doubled, as in bound).
    share = 0.0 if dtype == "f32" else 15.0 * scales.max() * sum(1000.0 * (g + 1) for g in range(K // group))
    assert_within(y, want, bound(want, mag, 3 * K + K // group + 2, dt) + 20 * 2.0 ** -23 * share)


def test_other_stream(ex):
    rng = np.random.default_rng(6)
    q, scales, _ = _weights(rng, 1, 512, 1024, 128, False)
    q, scales = torch.from_numpy(q[0]).cuda(), torch.from_numpy(scales[0]).cuda()
    x = torch.randn(4, 1024, device="cuda")
    want = ex.w4_matvec(x, q, scales, group=128)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = ex.w4_matvec(x, q, scales, group=128, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)


def test_refusals(ex):
    x = torch.zeros(2, 128, device="cuda")
    q = torch.zeros(3, 32, 64, dtype=torch.uint8, device="cuda")
    s = torch.zeros(3, 32, 1, device="cuda")
    ids = torch.zeros(2, dtype=torch.int32, device="cuda")
    with pytest.raises(ex.SgemmError):
        ex.w4_matvec(x, q, s, group=128)  # three matrices, no ids
    with pytest.raises(ex.SgemmError):
        ex.w4_matvec(x, q, s, group=512, ids=ids)  # unknown group size
    with pytest.raises(ValueError):
        ex.w4_matvec(x, q, s, group=64, ids=ids)  # scales of another group size
    with pytest.raises(ValueError):
        ex.w4_matvec(x[:, :64], q, s, group=128, ids=ids)
    with pytest.raises(TypeError):
        ex.w4_matvec(x, q, s, group=128, ids=ids.long())
    with pytest.raises(ValueError):
        ex.w4_matvec(x, q, s, group=128, ids=ids[:1])
    with pytest.raises(TypeError):
        ex.w4_matvec(x, q.to(torch.int8), s, group=128, ids=ids)
    with pytest.raises(ValueError):
        ex.w4_matvec(x, q, s, group=128, ids=ids, zeros=torch.zeros(3, 32, 2, dtype=torch.uint8, device="cuda"))

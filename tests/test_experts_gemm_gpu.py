"""Products per expert over ragged row groups, and the gradient of the experts' matrices, against 64-bit sums."""

import numpy as np
import pytest
import torch

from tests.experts_harness import (DTYPES, TINY, assert_within, bound, canaries_intact, offsets_of, strided)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ex():
    from dense_fp32_matrix_major_gb300 import experts

    return experts


def limit(exact, magnitude, terms, dt):
    """fp32 follows the library's product bound (1e-5 of the sum of magnitudes), the others the fp32 sum's."""
    if dt == torch.float32:
        return 1e-5 * magnitude + TINY[dt]
    return bound(exact, magnitude, terms, dt)


SHAPES = [
    # group sizes, rows after the last group, K, N
    ([1], 0, 1, 1), ([0], 3, 8, 8), ([5, 0, 1], 2, 64, 64), ([0, 0, 130, 0], 0, 128, 72), ([17, 300, 1, 64], 5, 96, 136),
    ([128, 256, 128], 0, 256, 256), ([255, 257, 1, 511], 0, 160, 384), ([33] * 9, 7, 40, 24), ([7, 90], 1, 33, 65),
    ([640], 0, 520, 264), ([3] * 40, 0, 192, 512), ([31, 65, 129], 3, 1537, 129), ([1000, 24], 0, 2056, 128),
]


def _inputs(rng, dt, counts, rest, K, N, trans):
    S, E = sum(counts) + rest, len(counts)
    a = torch.from_numpy(rng.standard_normal((S, K)).astype(np.float32)).to(dt)
    b = torch.from_numpy(rng.standard_normal((E, N, K) if trans else (E, K, N)).astype(np.float32)).to(dt)
    return a, b


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("counts,rest,K,N", SHAPES)
def test_gemm(ex, dtype, counts, rest, K, N, trans):
    dt = DTYPES[dtype]
    rng = np.random.default_rng(K * 7 + N)
    a, b = _inputs(rng, dt, counts, rest, K, N, trans)
    off = offsets_of(counts)
    S = a.shape[0]
    a64, b64 = a.double().numpy(), b.double().numpy()
    want, mag = np.zeros((S, N)), np.zeros((S, N))
    for e in range(len(counts)):
        rows = slice(int(off[e]), int(off[e + 1]))
        w = b64[e].T if trans else b64[e]
        want[rows], mag[rows] = a64[rows] @ w, np.abs(a64[rows]) @ np.abs(w)
    for pad, offset in ((0, 0), (8, 0), (3, 1)):
        out = strided(torch.zeros(S, N, dtype=dt), pad, offset)
        c = ex.gemm(strided(a, pad, offset), b.cuda(), off.cuda(), out=out, transB=trans)
        assert_within(c, want, limit(want, mag, K, dt), f"pad {pad}")
        assert canaries_intact(out)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("counts,rest,M,N", SHAPES)
def test_wgrad(ex, dtype, counts, rest, M, N):
    dt = DTYPES[dtype]
    rng = np.random.default_rng(M * 5 + N)
    S, E = sum(counts) + rest, len(counts)
    a = torch.from_numpy(rng.standard_normal((S, M)).astype(np.float32)).to(dt)
    b = torch.from_numpy(rng.standard_normal((S, N)).astype(np.float32)).to(dt)
    off = offsets_of(counts)
    a[int(off[-1]):] = float("nan")  # rows of no group are not read into a sum
    a64, b64 = a.double().numpy(), b.double().numpy()
    want, mag, terms = np.zeros((E, M, N)), np.zeros((E, M, N)), max(counts)
    for e in range(E):
        rows = slice(int(off[e]), int(off[e + 1]))
        want[e], mag[e] = a64[rows].T @ b64[rows], np.abs(a64[rows]).T @ np.abs(b64[rows])
    for pad, offset in ((0, 0), (8, 0), (1, 3)):
        out = strided(torch.full((E * M, N), 5.0, dtype=dt), pad, offset)
        view = out.as_strided((E, M, N), (M * out.stride(0), out.stride(0), 1), offset)
        ex.gemm_wgrad(strided(a, pad, offset), strided(b, pad, offset), off.cuda(), out=view)
        assert_within(view, want, limit(want, mag, terms, dt), f"pad {pad}")
        assert canaries_intact(out)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("counts,M,N", [
    ([5003], 64, 100), ([2, 0, 9001, 70], 40, 33), ([4096, 4095], 264, 72), ([0], 64, 64), ([7000], 1, 1),
])
def test_wgrad_of_long_groups(ex, dtype, counts, M, N):
    """Few small matrices summed over many rows: the sums are cut into slices of the rows."""
    dt = DTYPES[dtype]
    rng = np.random.default_rng(M * 3 + N)
    rest = 4000 if counts == [0] else 9
    S, E = sum(counts) + rest, len(counts)
    a = torch.from_numpy(rng.standard_normal((S, M)).astype(np.float32)).to(dt)
    b = torch.from_numpy(rng.standard_normal((S, N)).astype(np.float32)).to(dt)
    off = offsets_of(counts)
    b[int(off[-1]):] = float("inf")  # rows of no group are not read into a sum
    a64, b64 = a.double().numpy(), b.double().numpy()
    want, mag = np.zeros((E, M, N)), np.zeros((E, M, N))
    for e in range(E):
        rows = slice(int(off[e]), int(off[e + 1]))
        want[e], mag[e] = a64[rows].T @ b64[rows], np.abs(a64[rows]).T @ np.abs(b64[rows])
    for pad, offset in ((0, 0), (8, 0), (1, 3)):
        out = strided(torch.full((E * M, N), 5.0, dtype=dt), pad, offset)
        view = out.as_strided((E, M, N), (M * out.stride(0), out.stride(0), 1), offset)
        ex.gemm_wgrad(strided(a, pad, offset), strided(b, pad, offset), off.cuda(), out=view)
        assert_within(view, want, limit(want, mag, max(counts), dt), f"pad {pad}")
        assert canaries_intact(out)
        assert torch.equal(view, ex.gemm_wgrad(strided(a, pad, offset), strided(b, pad, offset), off.cuda()))
    if counts[0] > 100:  # an infinity and a NaN of one row reach its column of C alone, whatever its slice
        a[17, 3 % M], a[counts[0] - 1, 5 % M] = float("inf"), float("nan")
        g = ex.gemm_wgrad(a.cuda(), b.cuda(), off.cuda()).cpu()[0]
        touched = torch.zeros(M, dtype=torch.bool)
        touched[3 % M] = touched[5 % M] = True
        assert torch.isfinite(g[~touched]).all() and torch.isnan(g[5 % M]).all()
        assert M == 1 or torch.isinf(g[3]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("trans", [False, True])
def test_non_finite_values_stay_in_their_group(ex, dtype, trans):
    """NaN and infinities of one group's rows, of its neighbours' and of an empty group's matrix."""
    dt = DTYPES[dtype]
    counts, K, N = [40, 0, 37, 50], 72, 136
    rng = np.random.default_rng(3)
    a, b = _inputs(rng, dt, counts, 4, K, N, trans)
    off = offsets_of(counts)
    a[40:77] = float("nan")   # all of group 2
    a[5, 3] = float("inf")    # one row of group 0
    a[-4:] = float("nan")     # rows of no group
    b[1] = float("nan")       # the empty group's matrix
    c = ex.gemm(a.cuda(), b.cuda(), off.cuda(), transB=trans).cpu()
    assert torch.isnan(c[40:77]).all()
    assert (c[-4:] == 0).all()
    clean = torch.ones(c.shape[0], dtype=torch.bool)
    clean[5] = clean[-4:] = False
    clean[40:77] = False
    assert torch.isfinite(c[clean]).all()
    column = (b[0, :, 3] if trans else b[0, 3]).float()
    assert torch.equal(torch.sign(c[5].float()), torch.sign(column)) and torch.isinf(c[5]).all()
    g = ex.gemm_wgrad(a.cuda(), torch.ones(131, 64, dtype=dt, device="cuda"), off.cuda()).cpu()
    assert torch.isfinite(g[3]).all() and (g[1] == 0).all() and torch.isnan(g[2]).all()
    assert torch.isinf(g[0, 3]).all() and torch.isfinite(g[0, 4:]).all()


def test_gradients_against_differences(ex):
    """A product is linear in each factor: differences over a step of one equal the gradients."""
    rng = np.random.default_rng(11)
    counts, K, N = [33, 0, 70, 12], 48, 56
    S, E = sum(counts) + 3, len(counts)
    off = offsets_of(counts).cuda()

    def cuda(*shape):
        return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).cuda()

    def dot(x, y):
        return float((x.double() * y.double()).sum())

    for trans in (False, True):
        shape = (E, N, K) if trans else (E, K, N)
        a, u, b, v, dc = cuda(S, K), cuda(S, K), cuda(*shape), cuda(*shape), cuda(S, N)
        da = ex.gemm(dc, b, off, transB=not trans)
        db = ex.gemm_wgrad(dc, a, off) if trans else ex.gemm_wgrad(a, dc, off)
        # 1e-5 of the sum of magnitudes, in each of the products and over all outputs.
        tol = 1e-5 * S * K * N
        along_a = (dot(dc, ex.gemm(a + u, b, off, transB=trans)) - dot(dc, ex.gemm(a - u, b, off, transB=trans))) / 2
        along_b = (dot(dc, ex.gemm(a, b + v, off, transB=trans)) - dot(dc, ex.gemm(a, b - v, off, transB=trans))) / 2
        assert abs(along_a - dot(da, u)) <= tol
        assert abs(along_b - dot(db, v)) <= tol


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N", [104, 264])
def test_a_rows_result_is_its_own(ex, dtype, N, trans):
    """The same bits whatever rows a row is among, and however many: tiles are shaped by the sizes."""
    dt = DTYPES[dtype]
    rng = np.random.default_rng(17)
    counts, K = [700, 3, 650], 328
    a, b = _inputs(rng, dt, counts, 0, K, N, trans)
    a[10, 7], a[701, 5] = float("inf"), float("nan")
    a, b, off = a.cuda(), b.cuda(), offsets_of(counts)
    whole = ex.gemm(a, b, off.cuda(), transB=trans)
    for e in range(3):
        for first, few in ((0, 1), (1, 2), (counts[e] - 2, 2)):
            at = int(off[e]) + first
            part = ex.gemm(a[at:at + few], b[e:e + 1], offsets_of([few]).cuda(), transB=trans)
            assert torch.equal(torch.nan_to_num(part, 7.0), torch.nan_to_num(whole[at:at + few], 7.0))
            assert torch.equal(torch.isnan(part), torch.isnan(whole[at:at + few]))
    assert torch.isinf(whole[10]).all() and torch.isnan(whole[701]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_integer_values_are_exact(ex, dtype):
    dt = DTYPES[dtype]
    g = torch.Generator().manual_seed(2)
    counts = [300, 5, 0, 200]
    a = torch.randint(-2, 3, (505, 128), generator=g).to(dt)
    b = torch.randint(-2, 3, (4, 128, 256), generator=g).to(dt)
    off = offsets_of(counts)
    c = ex.gemm(a.cuda(), b.cuda(), off.cuda()).cpu().double()
    want = torch.cat([a[off[e]:off[e + 1]].double() @ b[e].double() for e in range(4)])
    assert want.abs().max() <= 256  # exact in bf16 too
    assert torch.equal(c, want)


def test_offsets_out_of_range_touch_nothing(ex):
    a, b = torch.ones(40, 64, device="cuda"), torch.ones(3, 64, 64, device="cuda")
    off = torch.tensor([0, -7, 1 << 30, 20], dtype=torch.int32, device="cuda")
    for dt in DTYPES.values():
        out = strided(torch.zeros(40, 64, dtype=dt), 0, 64)
        ex.gemm(a.to(dt), b.to(dt), off, out=out)
        assert canaries_intact(out)
        w = strided(torch.zeros(3 * 64, 64, dtype=dt), 0, 64)
        ex.gemm_wgrad(a.to(dt), a.to(dt), off, out=w.view(3, 64, 64))
        assert canaries_intact(w)


def test_other_stream(ex):
    a, b = torch.randn(500, 256, device="cuda"), torch.randn(4, 256, 384, device="cuda")
    off = offsets_of([100, 250, 0, 150]).cuda()
    want = ex.gemm(a, b, off)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = ex.gemm(a, b, off, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)


def test_refusals(ex):
    a, b = torch.zeros(8, 16, device="cuda"), torch.zeros(2, 16, 32, device="cuda")
    off = torch.tensor([0, 4, 8], dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        ex.gemm(a, b, off, transB=True)
    with pytest.raises(TypeError):
        ex.gemm(a, b.half(), off)
    with pytest.raises(ValueError):
        ex.gemm(a, b, off[:2])
    with pytest.raises(TypeError):
        ex.gemm(a, b, off.long())
    with pytest.raises(ValueError):
        ex.gemm(a, b, off, out=torch.zeros(8, 31, device="cuda"))
    with pytest.raises(ValueError):
        ex.gemm(a, b.transpose(1, 2), off, transB=True)
    with pytest.raises(ValueError):
        ex.gemm_wgrad(a, torch.zeros(7, 4, device="cuda"), off)
    with pytest.raises(ex.SgemmError):
        ex.gemm(a, b[:, :, :16], off, out=a)  # overlaps its input



@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_empty_sizes(ex, dtype):
    """No rows, no columns, nothing to sum, no tokens: results of the right shape, zeros where a sum is empty."""
    dt = DTYPES[dtype]

    def zeros(*shape):
        return torch.zeros(*shape, dtype=dt, device="cuda")

    off = torch.tensor([0, 0, 0], dtype=torch.int32, device="cuda")
    assert ex.gemm(zeros(0, 64), zeros(2, 64, 32), off).shape == (0, 32)
    assert ex.gemm(zeros(8, 64), zeros(2, 64, 0), off).shape == (8, 0)
    some = torch.tensor([0, 3, 8], dtype=torch.int32, device="cuda")
    for trans in (False, True):
        out = torch.ones(8, 32, dtype=dt, device="cuda")
        ex.gemm(zeros(8, 0), zeros(2, 32, 0) if trans else zeros(2, 0, 32), some, out=out, transB=trans)
        assert (out == 0).all()
    out = torch.ones(2, 64, 32, dtype=dt, device="cuda")
    ex.gemm_wgrad(zeros(0, 64), zeros(0, 32), off, out=out)
    assert (out == 0).all()
    assert ex.gemm_wgrad(zeros(8, 0), zeros(8, 32), some).shape == (2, 0, 32)
    r = ex.sort(torch.zeros(0, 2, dtype=torch.int64, device="cuda"), 2)
    assert r.offsets.tolist() == [0, 0, 0] and r.slot.shape == (0, 2) and r.order.shape == (0,)
    w = torch.zeros(0, 2, device="cuda")
    assert ex.gather(zeros(0, 16), r).shape == (0, 16) and ex.combine(zeros(0, 16), w, r).shape == (0, 16)
    dh, dw = ex.combine_grad(zeros(0, 16), zeros(0, 16), w, r)
    assert dh.shape == (0, 16) and dw.shape == (0, 2)
    r = ex.sort(torch.zeros(4, 2, dtype=torch.int64, device="cuda"), 2)
    w = torch.ones(4, 2, device="cuda")
    assert ex.gather(zeros(4, 0), r).shape == (8, 0) and ex.combine(zeros(8, 0), w, r).shape == (4, 0)
    dh, dw = ex.combine_grad(zeros(4, 0), zeros(8, 0), w, r)
    assert dh.shape == (8, 0) and (dw == 0).all()
    q, s = torch.zeros(32, 0, dtype=torch.uint8, device="cuda"), torch.zeros(32, 0, device="cuda")
    assert (ex.w4_matvec(zeros(3, 0), q, s, group=64) == 0).all()
    q, s = torch.zeros(0, 64, dtype=torch.uint8, device="cuda"), torch.zeros(0, 1, device="cuda")
    assert ex.w4_matvec(zeros(3, 128), q, s, group=128).shape == (3, 0)


def test_same_sign_sums(ex):
    """Long sums of one sign, where cut sums drift in one direction: fp32 within the library's bound."""
    g = torch.Generator(device="cuda").manual_seed(9)
    a = torch.rand((300, 4096), generator=g, device="cuda")
    b = torch.rand((2, 4096, 136), generator=g, device="cuda")
    off = torch.tensor([0, 170, 300], dtype=torch.int32, device="cuda")
    want = torch.cat([a[:170].double() @ b[0].double(), a[170:].double() @ b[1].double()])
    assert float(((ex.gemm(a, b, off).double() - want).abs() / want).max()) <= 1e-5
    d = torch.rand((300, 64), generator=g, device="cuda")
    want = torch.stack([a[:170].double().t() @ d[:170].double(), a[170:].double().t() @ d[170:].double()])
    assert float(((ex.gemm_wgrad(a, d, off).double() - want).abs() / want).max()) <= 1e-5


def test_no_wait_gives_up(ex):
    """The kernels' bounded waits report through sgemm_device_status, as the library's others do: none gave up."""
    from dense_fp32_matrix_major_gb300 import sgemm

    a, b = torch.randn(64, 128, device="cuda"), torch.randn(2, 128, 64, device="cuda")
    off = torch.tensor([0, 30, 64], dtype=torch.int32, device="cuda")
    ex.gemm(a, b, off)
    ex.gemm(a.bfloat16(), b.bfloat16(), off)
    assert sgemm.device_status() == 0

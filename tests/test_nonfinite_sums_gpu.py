"""NaN and infinities in long fp32 sums: the results are IEEE's, no bounded wait gives up on the way, and outputs that
a NaN among the inputs explains are not summed again."""

import pytest
import torch

from tests.experts_harness import offsets_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def libs():
    from dense_fp32_matrix_major_gb300 import experts, sgemm

    sgemm.set_variant("auto")
    sgemm.device_status()
    return experts, sgemm


def kinds(x):
    return torch.where(torch.isnan(x), 3, torch.where(torch.isposinf(x), 1, torch.where(torch.isneginf(x), 2, 0)))


def ms(f):
    f()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    f()
    b.record()
    b.synchronize()
    return a.elapsed_time(b)


@pytest.mark.parametrize("where", ["a", "b"])
def test_a_nan_row_of_a_long_group(libs, where):
    """One row of 49152 makes every entry of its group's gradient NaN, and only of its."""
    experts, sgemm = libs
    S, M, N = 49152, 2048, 2048
    a, b = torch.randn(S + 64, M, device="cuda"), torch.randn(S + 64, N, device="cuda")
    off = offsets_of([S, 64]).cuda()
    clean = experts.gemm_wgrad(a, b, off)
    (a if where == "a" else b)[S - 1] = float("nan")
    c = experts.gemm_wgrad(a, b, off)
    assert sgemm.device_status() == 0
    assert torch.isnan(c[0]).all()
    assert torch.equal(c[1], clean[1])


def test_time_of_a_nan_row(libs):
    """Sums that a NaN explains cost a look at the inputs each, not a serial sum per output (193 ms here)."""
    experts, _ = libs
    a, b = torch.randn(4096, 2048, device="cuda"), torch.randn(4096, 2048, device="cuda")
    off = offsets_of([4096]).cuda()
    b[4095] = float("nan")
    out = torch.empty(1, 2048, 2048, device="cuda")
    assert ms(lambda: experts.gemm_wgrad(a, b, off, out=out)) < 40


def plant(a, b):
    """Infinities and a NaN in factors S x M and S x N whose sums run over S, so that every IEEE rule decides some."""
    S = a.shape[0]
    a[5] = a[5].abs() + 1.0
    b[5, :300] = float("inf")              # inf times positive values
    b[S // 2, 7] = float("-inf")
    a[S // 2, ::3] = 0.0                   # -inf * 0
    a[S - 1, 11] = float("inf")
    b[S - 1, ::2] = b[S - 1, ::2].abs() + 0.5
    a[S - 3, 13] = float("nan")
    b[S // 3, 400] = float("nan")


@pytest.mark.parametrize("S,M,N", [(16384, 512, 2560), (4099, 1200, 1000), (8192, 130, 600)])
def test_infinities_of_long_sums(libs, S, M, N):
    experts, sgemm = libs
    g = torch.Generator(device="cuda").manual_seed(S)
    a, b = torch.randn((S, M), generator=g, device="cuda"), torch.randn((S, N), generator=g, device="cuda")
    plant(a, b)
    want = a.double().t() @ b.double()
    assert set(kinds(want).unique().tolist()) == {0, 1, 2, 3}
    fine = torch.isfinite(want)
    size = torch.nan_to_num(a, 0.0, 0.0, 0.0).abs().double().t() @ torch.nan_to_num(b, 0.0, 0.0, 0.0).abs().double()
    off = offsets_of([S]).cuda()
    at = a.t().contiguous()
    results = [experts.gemm_wgrad(a, b, off)[0], experts.gemm_wgrad(b, a, off)[0].t(),
               experts.gemm(at, b[None], offsets_of([M]).cuda()),
               experts.gemm(at, b.t().contiguous()[None], offsets_of([M]).cuda(), transB=True),
               sgemm.gemm(a, b, transA=True), sgemm.gemm(at, b)]
    assert sgemm.device_status() == 0
    for i, c in enumerate(results):
        assert torch.equal(kinds(c), kinds(want)), i
        assert ((c.double() - want).abs()[fine] <= 1e-5 * size[fine]).all(), i

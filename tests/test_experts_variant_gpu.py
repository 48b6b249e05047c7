"""fp32 products per expert follow sgemm_set_variant, as the library's other products do."""

import numpy as np
import pytest
import torch

from tests.experts_harness import offsets_of

pytestmark = pytest.mark.gpu


@pytest.fixture
def libs():
    from dense_fp32_matrix_major_gb300 import experts, sgemm

    yield experts, sgemm
    sgemm.set_variant("auto")


@pytest.mark.parametrize("trans", [False, True])
def test_ffma_products_are_fp32_products(libs, trans):
    """Sums of one product: the fp32 product, to the bit."""
    experts, sgemm = libs
    g = torch.Generator(device="cuda").manual_seed(3)
    a = torch.randn((70, 1), generator=g, device="cuda")
    b = torch.randn((2, 90, 1) if trans else (2, 1, 90), generator=g, device="cuda")
    off = offsets_of([30, 35]).cuda()
    want = torch.zeros(70, 90, device="cuda")
    for e, rows in enumerate((slice(0, 30), slice(30, 65))):
        want[rows] = a[rows] * b[e].reshape(1, 90)
    sgemm.set_variant("ffma")
    assert torch.equal(experts.gemm(a, b, off, transB=trans), want)
    assert sgemm.last_variant_used() == sgemm.SGEMM_FFMA
    one = torch.randn((2, 50), generator=g, device="cuda")
    other = torch.randn((2, 60), generator=g, device="cuda")
    db = experts.gemm_wgrad(one, other, offsets_of([1, 1]).cuda())
    assert torch.equal(db, one[:, :, None] * other[:, None])
    sgemm.set_variant("tf32x3")
    experts.gemm(a, b, off, transB=trans)
    assert sgemm.last_variant_used() == sgemm.SGEMM_TF32X3


def test_ffma_sums(libs):
    """Error of the fp32 sums themselves: at most 2^-24 of the magnitudes for each of K + 1 roundings."""
    experts, sgemm = libs
    g = torch.Generator(device="cuda").manual_seed(4)
    K, counts = 700, [65, 0, 200, 1]
    a, b = torch.randn((270, K), generator=g, device="cuda"), torch.randn((4, K, 130), generator=g, device="cuda")
    off = offsets_of(counts)
    sgemm.set_variant("ffma")
    c = experts.gemm(a, b, off.cuda())
    want, mag = torch.zeros_like(c, dtype=torch.float64), torch.zeros_like(c, dtype=torch.float64)
    for e in range(4):
        rows = slice(int(off[e]), int(off[e + 1]))
        want[rows], mag[rows] = a[rows].double() @ b[e].double(), a[rows].double().abs() @ b[e].double().abs()
    assert ((c.double() - want).abs() <= (K + 1) * 2.0 ** -24 * mag).all()
    d = experts.gemm_wgrad(a, c, off.cuda())
    for e, n in enumerate(counts):
        rows = slice(int(off[e]), int(off[e + 1]))
        want, mag = a[rows].double().t() @ c[rows].double(), a[rows].double().abs().t() @ c[rows].double().abs()
        assert ((d[e].double() - want).abs() <= (n + 1) * 2.0 ** -24 * mag).all()
    assert np.isfinite(d.cpu().numpy()).all()

"""The mixture-of-experts entry points without a GPU: the header and its binding agree, and bad arguments are
rejected before a device is touched."""

import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _header():
    with open(os.path.join(ROOT, "include", "experts.h")) as f:
        return re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)


@pytest.fixture(scope="module")
def ex():
    from dense_fp32_matrix_major_gb300 import _build

    _build.build()
    from dense_fp32_matrix_major_gb300 import experts

    return experts


def test_binding_covers_the_header(ex):
    names = set(re.findall(r"\b(sgemm_[a-z0-9_]+)\s*\(", _header()))
    assert len(names) == 8
    assert set(ex.SIGNATURES) == names
    for name, (_, args) in ex.SIGNATURES.items():
        declared = re.search(rf"\b{name}\s*\(([^;]*)\)\s*;", _header()).group(1)
        assert len(args) == declared.count(",") + 1, name


def test_constants_match_the_header(ex):
    text = _header()
    for name, value in re.findall(r"\b(SGEMM_[A-Z0-9_]+)\s*=\s*(-?\d+)", text):
        assert getattr(ex, name) == int(value), name
    for name, value in re.findall(r"#define\s+(SGEMM_[A-Z0-9_]+)\s+(\d+)", text):
        assert getattr(ex, name) == int(value), name


def test_sort_workspace(ex):
    f = ex.lib.sgemm_experts_sort_workspace
    assert f(0, 8) == 0 and f(64, 8) == 0
    assert f(1 << 20, 256) % (257 * 4) == 0 and f(1 << 20, 256) > 0
    assert f(-1, 8) == 0 and f(64, 0) == 0 and f(64, ex.SGEMM_EXPERTS_MAX + 1) == 0


P = 0x100000  # addresses far apart; never read


@pytest.mark.parametrize("change", [
    {"id_bits": 16}, {"tokens": -1}, {"top_k": 0}, {"top_k": 65}, {"experts": 0}, {"experts": 4097},
    {"ids": 0}, {"offsets": 0}, {"order": 0}, {"slot": 0}, {"ids": 2 * P + 8}, {"order": 4 * P}, {"ids": P + 1},
    {"tokens": 1 << 30, "top_k": 2}, {"tokens": 1 << 16}, {"tokens": 1 << 16, "ws": 6 * P, "ws_bytes": 16},
])
def test_sort_refuses(ex, change):
    a = {"ids": P, "id_bits": 32, "tokens": 8, "top_k": 2, "experts": 4, "offsets": 2 * P, "order": 3 * P,
         "slot": 4 * P, "ws": 0, "ws_bytes": 0}
    a.update(change)
    assert ex.lib.sgemm_experts_sort(*a.values(), None) == 1


def _rows_args():
    return {"type": 0, "tokens": 8, "top_k": 2, "experts": 4, "width": 64}


@pytest.mark.parametrize("change", [
    {"type": 3}, {"type": -1}, {"tokens": -1}, {"top_k": 0}, {"experts": 0}, {"width": -1}, {"ldx": 63}, {"ldo": 63},
    {"x": 0}, {"slot": 0}, {"offsets": 0}, {"out": 0}, {"x": P + 2}, {"out": P + 128}, {"out": 2 * P - 64},
    {"ldx": 1 << 60},
])
def test_gather_and_combine_refuse(ex, change):
    a = {**_rows_args(), "x": P, "ldx": 64, "slot": 2 * P, "offsets": 3 * P, "out": 4 * P, "ldo": 64}
    a.update(change)
    assert ex.lib.sgemm_experts_gather(*a.values(), None) == 1
    head = [a[k] for k in ("type", "tokens", "top_k", "experts", "width", "x", "ldx")]
    tail = [a[k] for k in ("slot", "offsets", "out", "ldo")]
    for weights in (0, 5 * P):
        assert ex.lib.sgemm_experts_combine(*head, weights, *tail, None) == 1


@pytest.mark.parametrize("change", [
    {"type": 5}, {"lddy": 1}, {"ldh": 1}, {"lddh": 1}, {"weights": 0}, {"dweights": 0}, {"dh": 2 * P}, {"dh": P},
    {"dweights": 3 * P}, {"dh": 7 * P - 4},
])
def test_combine_grad_refuses(ex, change):
    a = {**_rows_args(), "dy": P, "lddy": 64, "h": 2 * P, "ldh": 64, "weights": 3 * P, "slot": 4 * P,
         "offsets": 5 * P, "dh": 6 * P, "lddh": 64, "dweights": 7 * P}
    a.update(change)
    assert ex.lib.sgemm_experts_combine_grad(*a.values(), None) == 1


@pytest.mark.parametrize("change", [
    {"type": 3}, {"trans": 2}, {"rows": -1}, {"rows": 1 << 31}, {"N": -1}, {"K": -1}, {"experts": 0},
    {"experts": 5000}, {"offsets": 0}, {"A": 0}, {"B": 0}, {"C": 0}, {"lda": 15}, {"ldb": 31}, {"ldc": 31},
    {"strideB": 511}, {"strideB": -512}, {"C": P}, {"C": 2 * P + 64}, {"C": 4 * P + 4}, {"A": P + 2},
])
def test_gemm_refuses(ex, change):
    a = {"type": 0, "trans": 0, "rows": 8, "N": 32, "K": 16, "experts": 4, "offsets": 4 * P, "A": P, "lda": 16,
         "B": 2 * P, "ldb": 32, "strideB": 512, "C": 3 * P, "ldc": 32}
    a.update(change)
    assert ex.lib.sgemm_experts_gemm(*a.values(), None) == 1


@pytest.mark.parametrize("change", [
    {"type": 3}, {"rows": -1}, {"M": -1}, {"N": -1}, {"experts": 0}, {"offsets": 0}, {"A": 0}, {"B": 0}, {"C": 0},
    {"lda": 15}, {"ldb": 31}, {"ldc": 31}, {"strideC": 511}, {"C": P}, {"C": 2 * P}, {"C": 4 * P},
])
def test_gemm_wgrad_refuses(ex, change):
    a = {"type": 0, "rows": 8, "M": 16, "N": 32, "experts": 4, "offsets": 4 * P, "A": P, "lda": 16, "B": 2 * P,
         "ldb": 32, "C": 3 * P, "ldc": 32, "strideC": 512}
    a.update(change)
    assert ex.lib.sgemm_experts_gemm_wgrad(*a.values(), None) == 1


def test_most_rows(ex):
    """Rows near 2^31 are refused by their number alone: nothing else is wrong here, and nothing to do."""
    for rows, refused in (((1 << 31) - 1025, False), ((1 << 31) - 1024, True)):
        assert (ex.lib.sgemm_experts_gemm(0, 0, rows, 0, 0, 4, 4 * P, 0, 1, 0, 1, 0, 0, 1, None) == 1) == refused
        assert (ex.lib.sgemm_experts_gemm_wgrad(0, rows, 0, 0, 4, 4 * P, 0, 1, 0, 1, 0, 1, 0, None) == 1) == refused


@pytest.mark.parametrize("change", [
    {"type": 3}, {"rows": -1}, {"rows": 65536}, {"N": -1}, {"K": 63}, {"group": 48}, {"group": 0}, {"group": 512},
    {"experts": 0}, {"ids": 0}, {"x": 0}, {"q": 0}, {"scales": 0}, {"scale_type": 3}, {"y": 0}, {"ldx": 63},
    {"ldy": 31}, {"y": P}, {"y": 2 * P}, {"y": 3 * P}, {"y": 4 * P}, {"y": 6 * P}, {"x": P + 2}, {"scales": 3 * P + 2},
])
def test_w4_matvec_refuses(ex, change):
    a = {"type": 0, "rows": 2, "N": 32, "K": 64, "group": 32, "experts": 4, "ids": 6 * P, "x": P, "ldx": 64,
         "q": 2 * P, "scales": 3 * P, "scale_type": 0, "zeros": 4 * P, "y": 5 * P, "ldy": 32}
    a.update(change)
    assert ex.lib.sgemm_w4_matvec(*a.values(), None) == 1


def test_python_checks_come_before_the_library(ex):
    import torch

    r = ex.Routing(torch.zeros(5, dtype=torch.int32), torch.zeros(4, dtype=torch.int32),
                   torch.zeros(2, 2, dtype=torch.int32))
    with pytest.raises(TypeError):
        ex.sort(torch.zeros(2, 2, dtype=torch.int32), 4)  # not on the GPU
    with pytest.raises(TypeError):
        ex.gather(torch.zeros(2, 8), r)
    with pytest.raises(TypeError):
        ex.gather(torch.zeros(2, 8, dtype=torch.float64), r)
    with pytest.raises(TypeError):
        ex.combine(torch.zeros(4, 8), None, r)
    with pytest.raises(TypeError):
        ex.gemm(torch.zeros(4, 8), torch.zeros(4, 8, 8), r.offsets)
    with pytest.raises(TypeError):
        ex.w4_matvec(torch.zeros(1, 64), torch.zeros(8, 32, dtype=torch.uint8), torch.zeros(8, 2), group=32)

"""The 8-bit operators and the layer for a few tokens without a GPU: headers and bindings agree, bad arguments are
rejected before a device is touched, every tensor's device is checked."""

import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _header(name):
    with open(os.path.join(ROOT, "include", name)) as f:
        return re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)


@pytest.fixture(scope="module")
def mods():
    from dense_fp32_matrix_major_gb300 import _build

    _build.build()
    from dense_fp32_matrix_major_gb300 import fp8, layer

    return {"fp8.h": fp8, "layer.h": layer}


@pytest.fixture(scope="module")
def lib(mods):
    return mods["fp8.h"].lib


@pytest.mark.parametrize("name,count", [("fp8.h", 4), ("layer.h", 2)])
def test_bindings_cover_the_headers(mods, name, count):
    mod, text = mods[name], _header(name)
    names = set(re.findall(r"\b(sgemm_[a-z0-9_]+)\s*\(", text))
    assert len(names) == count and set(mod.SIGNATURES) == names
    for fn, (_, args) in mod.SIGNATURES.items():
        declared = re.search(rf"\b{fn}\s*\(([^;]*)\)\s*;", text).group(1)
        assert len(args) == declared.count(",") + 1, fn
    for key, value in re.findall(r"\b(SGEMM_[A-Z0-9_]+)\s*=\s*(-?\d+)", text) + \
            re.findall(r"#define\s+(SGEMM_[A-Z0-9_]+)\s+(\d+)", text):
        assert getattr(mod, key) == int(value), key


def test_blocks_of_groups(lib):
    f = lib.sgemm_fp8_blocks
    assert [f(0, 4), f(1, 4), f(3, 4), f(128, 1), f(129, 1), f(1000, 16)] == [0, 1, 3, 1, 2, 23]
    assert f(-1, 4) == 0 and f(5, 0) == 0 and f(5, 4097) == 0
    # No cut of the rows into groups needs more.
    for rows, counts in ((4, [1, 1, 2]), (258, [129, 129]), (384, [127, 129, 128])):
        assert sum(-(-c // 128) for c in counts) <= f(rows, len(counts))


P = 0x1000000  # addresses far apart; never read


@pytest.mark.parametrize("change", [
    {"type": 3}, {"type": -1}, {"block": 3}, {"block": -1}, {"to": 2}, {"items": -1}, {"rows": -1}, {"cols": -1},
    {"items": 2}, {"block": 1, "items": 2}, {"x": 0}, {"x": P + 2}, {"q": 0}, {"scales": 0}, {"scales": 3 * P + 2},
    {"ldx": 255}, {"ldq": 255}, {"offsets": 4 * P}, {"block": 2, "offsets": 4 * P}, {"experts": 0}, {"experts": 2},
    {"block": 1, "offsets": 4 * P + 2}, {"q": P + 64}, {"scales": P + 64}, {"scales": 2 * P}, {"rows": 1 << 31},
    {"block": 1, "experts": 5000, "offsets": 4 * P}, {"block": 1, "experts": 4, "offsets": 2 * P + 32},
    {"block": 2, "items": 2, "strideX": 100}, {"block": 2, "items": 2, "strideX": 1 << 20, "strideQ": 100},
    {"ldx": 1 << 58},
])
def test_quantize_refuses(lib, change):
    a = {"type": 0, "block": 0, "to": 0, "pow2": 0, "items": 1, "rows": 16, "cols": 256, "x": P, "ldx": 256,
         "strideX": 0, "experts": 1, "offsets": 0, "q": 2 * P, "ldq": 256, "strideQ": 0, "scales": 3 * P}
    a.update(change)
    assert lib.sgemm_fp8_quantize(*a.values(), None) == 1


@pytest.mark.parametrize("change", [
    {"out": 3}, {"trans": 2}, {"ta": 2}, {"tb": -1}, {"rows": -1}, {"N": -1}, {"K": -1}, {"K": 1 << 31},
    {"experts": 0}, {"experts": 2}, {"A": 0}, {"A": P + 8}, {"lda": 264}, {"lda": 128}, {"sA": 0}, {"B": 0},
    {"B": 3 * P + 1}, {"ldb": 248}, {"ldb": 260}, {"sB": 0}, {"sB": 4 * P + 2}, {"C": 0}, {"C": 5 * P + 2},
    {"ldc": 63}, {"C": P + 64}, {"C": 3 * P + 64}, {"C": 2 * P}, {"C": 4 * P}, {"offsets": 5 * P},
    {"experts": 2, "offsets": 6 * P, "strideB": 100}, {"experts": 2, "offsets": 6 * P, "strideB": 16392},
    {"experts": 5000, "offsets": 6 * P, "strideB": 1 << 15}, {"offsets": 6 * P + 2}, {"rows": (1 << 31) - 1},
])
def test_gemm_refuses(lib, change):
    a = {"out": 0, "trans": 1, "ta": 0, "tb": 0, "rows": 32, "N": 64, "K": 256, "experts": 1, "offsets": 0, "A": P,
         "lda": 256, "sA": 2 * P, "B": 3 * P, "ldb": 256, "strideB": 0, "sB": 4 * P, "C": 5 * P, "ldc": 64}
    a.update(change)
    assert lib.sgemm_fp8_gemm(*a.values(), None) == 1


@pytest.mark.parametrize("change", [
    {"out": 3}, {"ta": 2}, {"tb": 2}, {"rows": -1}, {"M": -1}, {"N": -1}, {"experts": 0}, {"experts": 2}, {"A": 0},
    {"A": P + 8}, {"lda": 72}, {"lda": 48}, {"sA": 0}, {"B": 0}, {"ldb": 100}, {"sB": 0}, {"C": 0}, {"C": 5 * P + 1},
    {"ldc": 31}, {"C": P}, {"C": 2 * P}, {"C": 3 * P + 64}, {"C": 4 * P}, {"offsets": 6 * P, "rows": 130},
    {"offsets": 6 * P, "experts": 2, "strideC": 100}, {"offsets": 5 * P}, {"M": 1 << 31},
])
def test_wgrad_refuses(lib, change):
    a = {"out": 0, "ta": 0, "tb": 0, "rows": 256, "M": 64, "N": 32, "experts": 1, "offsets": 0, "A": P, "lda": 64,
         "sA": 2 * P, "B": 3 * P, "ldb": 32, "sB": 4 * P, "C": 5 * P, "ldc": 32, "strideC": 0}
    a.update(change)
    assert lib.sgemm_fp8_gemm_wgrad(*a.values(), None) == 1


@pytest.mark.parametrize("change", [
    {"type": 3}, {"held": 3}, {"held": -1}, {"act": 4}, {"act": -1}, {"tokens": -1}, {"top_k": 0}, {"top_k": 65},
    {"tokens": 257}, {"experts": 0}, {"experts": 4097}, {"width": -1}, {"hidden": -1}, {"hidden": 1 << 25},
    {"x": 0}, {"x": P + 1}, {"ldx": 63}, {"ids": 0}, {"ids": 2 * P + 2}, {"id_bits": 16}, {"weights": 0}, {"w1": 0},
    {"ld1": 63}, {"stride1": 4000}, {"w2": 0}, {"ld2": 31}, {"stride2": 2000}, {"y": 0}, {"ldy": 63}, {"ws": 0},
    {"ws": 9 * P + 8}, {"bytes": 16}, {"y": P}, {"y": 4 * P + 64}, {"ws": 6 * P}, {"y": 9 * P},
    {"held": 1}, {"held": 1, "s1": 5 * P, "s2": 7 * P, "ld1": 72, "stride1": 64 * 72},
    {"held": 1, "s1": 5 * P, "s2": 7 * P, "w2": 6 * P + 4},
])
def test_layer_refuses(lib, change):
    a = {"type": 0, "held": 0, "act": 3, "gated": 1, "tokens": 4, "top_k": 2, "experts": 4, "width": 64, "hidden": 32,
         "x": P, "ldx": 64, "ids": 2 * P, "id_bits": 32, "weights": 3 * P, "w1": 4 * P, "ld1": 64, "stride1": 4096,
         "s1": 0, "w2": 6 * P, "ld2": 32, "stride2": 2048, "s2": 0, "y": 8 * P, "ldy": 64, "ws": 9 * P, "bytes": 1 << 20}
    a.update(change)
    assert lib.sgemm_experts_layer(*a.values(), None) == 1


def test_layer_workspace(lib):
    f = lib.sgemm_experts_layer_workspace
    assert f(0, 2, 64) == 0 and f(4, 2, 64) == 8 * 64 * 4 and f(4, 2, 65) == 8 * 72 * 4
    assert f(257, 2, 64) == 0 and f(-1, 2, 64) == 0 and f(4, 0, 64) == 0 and f(4, 2, -1) == 0


class Stop(Exception):
    pass


def test_calls_check_every_tensor(mods, monkeypatch):
    """Each call hands all its tensors to the device check, outputs, scales and offsets among them."""
    fp8, layer = mods["fp8.h"], mods["layer.h"]
    seen = []

    def check(stream, *tensors):
        seen.append(tensors)
        raise Stop

    for mod in (fp8, layer):
        monkeypatch.setattr(mod, "_stream_handle", check)
        monkeypatch.setattr(mod, "_contiguous", lambda t, *rest: 0)
        monkeypatch.setattr(mod, "_strides", lambda t, *rest: (16, 16))
    monkeypatch.setattr(layer, "_rows", lambda t, *rest: (0, t.shape[1]))

    def q(*shape):
        return fp8.Quantized(torch.zeros(shape, dtype=torch.float8_e4m3fn), torch.zeros(1))

    x, off = torch.zeros(128, 16), torch.zeros(3, dtype=torch.int32)
    a, b, c, g = q(128, 16), q(2, 32, 16), torch.zeros(128, 32), torch.zeros(2, 16, 32)
    out = q(256, 16)
    ids, w, y = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2), torch.zeros(4, 16)
    w1, w2 = q(2, 64, 16), q(2, 16, 32)
    monkeypatch.setattr(fp8, "_operand", lambda t, *rest: (0, 16, 16, 0, 0))
    for call, tensors in (
        (lambda: fp8.quantize(x, "columns", offsets=off, out=out), (x, off, *out)),
        (lambda: fp8.gemm(a, b, off, out=c, transB=True), (*a, *b, off, c)),
        (lambda: fp8.gemm_wgrad(a, q(128, 32), off, out=g), (*a, off, g)),
        (lambda: layer.forward(y, ids, w, w1, w2, gated=True, out=torch.zeros(4, 16)),
         (y, ids, w, w1.values, w1.scales, w2.values, w2.scales)),
    ):
        with pytest.raises(Stop):
            call()
        got = seen.pop()
        assert all(any(t is g_ for g_ in got) for t in tensors)


def test_binding_refuses_what_does_not_fit(mods):
    fp8, layer = mods["fp8.h"], mods["layer.h"]
    x = torch.zeros(4, 16)
    with pytest.raises(ValueError):
        fp8.quantize(x, "tiles")
    with pytest.raises(TypeError):
        fp8.quantize(x, "rows", dtype=torch.int8)
    with pytest.raises(TypeError):
        fp8.quantize(x, "rows")  # not on a GPU
    with pytest.raises(TypeError):
        fp8.gemm(x, x)
    with pytest.raises(TypeError):
        layer.forward(x, torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2), x, x)

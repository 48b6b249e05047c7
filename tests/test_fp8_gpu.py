"""Quantisation to 8-bit floating point and products of 8-bit matrices, against definitions in 64 bits."""

import numpy as np
import pytest
import torch

from tests.experts_harness import DTYPES, ROUNDING, TINY, canaries_intact, offsets_of, strided
from tests.fp8_harness import E4M3, E5M2, LARGEST, check_product, meaning, quantize64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fp8():
    from dense_fp32_matrix_major_gb300 import fp8

    return fp8


@pytest.fixture(autouse=True)
def no_wait_gave_up():
    yield
    from dense_fp32_matrix_major_gb300 import sgemm

    torch.cuda.synchronize()
    assert sgemm.device_status() == 0


def same(got, want):
    got = got.double().cpu().numpy()
    assert got.shape == want.shape
    assert np.array_equal(got, want, equal_nan=True), f"{(got != want).sum()} of {got.size} differ"


def rows_of(rows, cols, dtype, seed=0, spread=2.0):
    g = torch.Generator().manual_seed(seed + 1000 * rows + cols)
    x = torch.randn((rows, cols), generator=g) * torch.exp(spread * torch.randn((rows, 1), generator=g))
    return x.to(dtype)


# ------------------------------------------------------------------ quantisation


@pytest.mark.parametrize("block", ["rows", "columns", "blocks"])
@pytest.mark.parametrize("name", list(DTYPES))
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 127), (5, 128), (130, 129), (257, 515), (128, 512), (2, 1040)])
def test_quantize(fp8, block, name, rows, cols):
    x = rows_of(rows, cols, DTYPES[name])
    for to in (E4M3, E5M2):
        for pow2 in (False, True):
            q = fp8.quantize(x.cuda(), block, dtype=to, pow2=pow2)
            values, scales = quantize64(x, block, to, pow2)
            same(q.values, values)
            same(q.scales, scales.astype(np.float64))
            assert q.values.stride(0) % 16 == 0 or rows == 1


@pytest.mark.parametrize("block", ["rows", "columns", "blocks"])
@pytest.mark.parametrize("pad,offset", [(0, 0), (1, 0), (0, 1), (7, 3), (8, 8)])
def test_quantize_strides(fp8, block, pad, offset):
    for name, dtype in DTYPES.items():
        x = strided(rows_of(70, 260, dtype), pad, offset)
        store = torch.full((70 * 300 + 40,), 0x5A, dtype=torch.uint8, device="cuda")
        out = store.view(E4M3).as_strided((70, 260), (260 + pad, 1), offset)
        want = fp8.quantize(x.contiguous(), block)
        got = fp8.quantize(x, block, out=fp8.Quantized(out, torch.empty_like(want.scales)))
        assert torch.equal(got.values.view(torch.uint8), want.values.view(torch.uint8)), name
        assert torch.equal(got.scales, want.scales)
        out.view(torch.uint8).fill_(0x5A)
        assert bool((store == 0x5A).all()) and canaries_intact(x.copy_(x))


def test_quantize_a_stack(fp8):
    x = torch.stack([rows_of(130, 200, torch.float32, s) for s in range(3)])
    q = fp8.quantize(x.cuda(), "blocks")
    assert q.values.shape == (3, 130, 200) and q.scales.shape == (3, 2, 2)
    for i in range(3):
        values, scales = quantize64(x[i], "blocks", E4M3)
        same(q.values[i], values)
        same(q.scales[i], scales.astype(np.float64))
    part = fp8.quantize(x.cuda()[:, 5:100], "blocks")  # items further apart than they are long
    assert torch.equal(part.scales[1], fp8.quantize(x[1, 5:100].contiguous().cuda(), "blocks").scales)


@pytest.mark.parametrize("block", ["rows", "columns", "blocks"])
def test_quantize_special_values(fp8, block):
    """Zeros, the smallest and largest numbers, infinities and NaN."""
    x = rows_of(140, 260, torch.float32, 5)
    x[0:128, 0:128] = 0.0
    x[3, 200] = float("inf")
    x[4, 201] = float("-inf")
    x[5, 202] = float("nan")
    x[130, :] = torch.linspace(-1e-38, 1e-38, 260)
    x[131, 0:128] = 3e38
    x[132, :] = float("nan")
    x[133, 5] = -0.0
    x[134, :] = float("inf")
    x[135, :] = 1e-45
    for to in (E4M3, E5M2):
        for pow2 in (False, True):
            q = fp8.quantize(x.cuda(), block, dtype=to, pow2=pow2)
            values, scales = quantize64(x, block, to, pow2)
            same(q.values, values)
            same(q.scales, scales.astype(np.float64))
            assert bool(torch.isfinite(q.scales).all()) and bool((q.scales >= 2.0 ** -126).all())


@pytest.mark.parametrize("name", ["bf16", "f16"])
@pytest.mark.parametrize("pad", [0, 1])
@pytest.mark.parametrize("block", ["rows", "columns", "blocks"])
def test_quantize_special_values_of_16_bits(fp8, block, pad, name):
    """The same, in rows that are 16-byte aligned and in others."""
    dtype = DTYPES[name]
    big, small = torch.finfo(dtype).max, torch.finfo(dtype).smallest_normal
    x = rows_of(300, 264, dtype, 6)
    x[0:128, 0:128] = 0.0
    x[3, 200] = float("inf")
    x[4, 201] = float("-inf")
    x[5, 202] = float("nan")
    x[6, 203] = -float("nan")
    x[128:256, 5] = float("nan")
    x[130, :] = torch.linspace(-small, small, 264)
    x[131, 0:64] = big
    x[132, :] = float("nan")
    x[133, 5] = -0.0
    x[134, :] = float("inf")
    x[256:, 128:256] = float("-inf")
    x[299, 130] = -big
    room = torch.zeros((300, 264 + pad), dtype=dtype, device="cuda")
    room[:, :264] = x.cuda()
    for to in (E4M3, E5M2):
        q = fp8.quantize(room[:, :264], block, dtype=to)
        values, scales = quantize64(x, block, to)
        same(q.values, values)
        same(q.scales, scales.astype(np.float64))


def test_quantize_every_border(fp8):
    """All 8-bit values, the borders between them and their neighbours in fp32, at a scale of 1."""
    for to in (E4M3, E5M2):
        v = torch.arange(127 if to == E4M3 else 124, dtype=torch.uint8).view(to).float()
        mid = (v[1:] + v[:-1]) / 2
        near = torch.cat([v, mid, torch.nextafter(mid, mid + 1), torch.nextafter(mid, mid - 1)])
        near = torch.cat([near, -near])
        x = torch.zeros((near.numel(), 128))
        x[:, 0], x[:, 1] = LARGEST[to], near
        q = fp8.quantize(x.cuda(), "rows", dtype=to)
        same(q.values, quantize64(x, "rows", to)[0])
        assert bool((q.scales == 1).all())


def test_quantize_against_the_quotient(fp8):
    """x times the rounded reciprocal of the scale, two roundings of 2^-24, against x / scale rounded once to 8 bits: the
    same but where the quotient lies within 2^-23 (and the roundings' product) of a border between two 8-bit values."""
    g = torch.Generator().manual_seed(21)
    for to in (E4M3, E5M2):
        v = torch.arange(127 if to == E4M3 else 124, dtype=torch.uint8).view(to).double()
        x = torch.randn((400, 128), generator=g, dtype=torch.float64)
        scale = torch.exp(3 * torch.randn((400, 1), generator=g, dtype=torch.float64))
        at = torch.randint(1, len(v) - 1, (400, 127), generator=g)
        close = (v[at] + v[at + 1]) / 2 * (1 + torch.randint(-4, 5, at.shape, generator=g) * 2.0 ** -24)
        x[:, 1:] = torch.where(torch.rand(at.shape, generator=g) < 0.7, close * x[:, 1:].sign(), x[:, 1:])
        x[:, 0] = LARGEST[to]
        x = (x * scale).float()
        q = fp8.quantize(x.cuda(), "rows", dtype=to)
        t = x.double() / q.scales.cpu().double().t()
        codes = v.numpy()
        want = codes[np.abs(np.abs(t.numpy())[..., None] - codes).argmin(-1)] * np.sign(t.numpy())
        got = q.values.double().cpu().numpy()
        differ = got != want
        border = (got[differ] + want[differ]) / 2
        assert (np.abs(t.numpy()[differ] - border) <= 2.0 ** -23 * (1 + 2.0 ** -20) * np.abs(border)).all()
        assert 0 < differ.mean() < 0.3


def reference8(x, block, to):
    """Values (as bytes) and scales of finite x, whole blocks at a time: PyTorch's fp32 arithmetic and cast."""
    high, wide = {"rows": (1, 128), "columns": (128, 1), "blocks": (128, 128)}[block]
    R, C = x.shape[-2:]
    t = torch.nn.functional.pad(x.float(), (0, -C % wide, 0, -R % high))
    t = t.reshape(*x.shape[:-2], t.shape[-2] // high, high, t.shape[-1] // wide, wide)
    most = t.abs().amax((-3, -1), keepdim=True)
    s = (most / torch.full_like(most, LARGEST[to])).clamp(min=2.0 ** -126)  # (a number's reciprocal would be rounded first)
    q = (t * (1 / s)).to(to).view(torch.uint8)
    s = s[..., 0, :, 0]
    return (q.reshape(*x.shape[:-2], q.shape[-4] * high, -1)[..., :R, :C],
            (s.transpose(-1, -2) if block == "rows" else s).contiguous())


@pytest.mark.parametrize("name", list(DTYPES))
@pytest.mark.parametrize("block,shape", [("columns", (6001, 2600)), ("blocks", (6001, 2600)), ("blocks", (11, 900, 1300)),
                                         ("rows", (6001, 2600))], ids=str)
def test_quantize_many_tiles(fp8, name, block, shape):
    """More tiles than blocks of threads are resident, so that each takes several."""
    g = torch.Generator(device="cuda").manual_seed(5)
    x = (torch.randn(shape, generator=g, device="cuda") * torch.exp(torch.randn(shape[-1:], generator=g, device="cuda")))
    x = x.to(DTYPES[name])
    for to in (E4M3, E5M2):
        q = fp8.quantize(x, block, dtype=to)
        values, scales = reference8(x, block, to)
        assert torch.equal(q.values.view(torch.uint8), values) and torch.equal(q.scales, scales)


@pytest.mark.parametrize("name", list(DTYPES))
def test_quantize_many_tiles_in_groups(fp8, name):
    g = torch.Generator(device="cuda").manual_seed(6)
    counts = [300, 0, 1, 128, 129, 700, 0, 513] * 5
    rows, cols = sum(counts) + 77, 2600
    x = torch.randn((rows, cols), generator=g, device="cuda").to(DTYPES[name])
    q = fp8.quantize(x, "columns", offsets=offsets_of(counts).cuda())
    at = first = 0
    for n in counts:
        if n:
            values, scales = reference8(x[first:first + n], "columns", E4M3)
            whole = len(scales) * 128
            assert torch.equal(q.values[at:at + n].view(torch.uint8), values)
            assert not q.values[at + n:at + whole].view(torch.uint8).any()
            assert torch.equal(q.scales[at // 128:at // 128 + len(scales)], scales)
            at, first = at + whole, first + n
    assert not q.values[at:].view(torch.uint8).any() and bool((q.scales[at // 128:] == 2.0 ** -126).all())


@pytest.mark.parametrize("counts,tail", [([5, 0, 128, 129, 0], 0), ([300], 7), ([0, 0, 0], 3), ([1] * 40, 0),
                                         ([128, 128], 0), ([0] * 100 + [1, 200], 50)])
def test_quantize_groups(fp8, counts, tail):
    rows, cols = sum(counts) + tail, 200
    x = rows_of(rows, cols, torch.bfloat16)
    q = fp8.quantize(x.cuda(), "columns", dtype=E5M2, offsets=offsets_of(counts).cuda())
    at, values, scales = 0, [], []
    for c in counts:
        v, s = quantize64(x[at:at + c], "columns", E5M2)
        at += c
        values += [v, np.zeros((-c % 128, cols))]
        scales.append(s)
    values, scales = np.concatenate(values), np.concatenate(scales)
    blocks = (rows + 127 * min(rows, len(counts))) // 128
    assert q.values.shape == (128 * blocks, cols) and q.scales.shape == (blocks, cols)
    n = scales.shape[0]
    same(q.values[:128 * n], values)
    same(q.scales[:n], scales.astype(np.float64))
    assert not q.values[128 * n:].view(torch.uint8).any() and bool((q.scales[n:] == 2.0 ** -126).all())


def test_quantize_groups_of_bad_offsets(fp8):
    """Offsets past the rows or that decrease are limited: no row is read from outside."""
    x = rows_of(300, 130, torch.float32).cuda()
    for off in ([0, 1000, 2000], [0, -5, 300], [0, 200, 100], [7, 8, 9]):
        q = fp8.quantize(x, "columns", offsets=torch.tensor(off, dtype=torch.int32, device="cuda"))
        assert bool(torch.isfinite(q.scales).all())


def limited(off, rows):
    """The groups that offsets stand for, and the first row behind them: bounds limited to 0 .. rows, the first taken as
    0, a group that would end before it starts empty."""
    o = [0] + [min(max(i, 0), rows) for i in off[1:]]
    return [(b, max(b, e)) for b, e in zip(o, o[1:])], o[-1]


BAD_OFFSETS = [[0, 1000, 2000], [0, -5, 300], [0, 200, 100], [7, 8, 9], [0, 2 ** 31 - 1, -2 ** 31], [0, 150, 20, 290],
               [5, 100, 100, 2 ** 31 - 1]]


@pytest.mark.parametrize("off", BAD_OFFSETS, ids=str)
@pytest.mark.parametrize("name", ["f32", "bf16"])
def test_quantize_groups_of_limited_offsets(fp8, off, name):
    """Offsets past the rows, below zero or decreasing give the groups that they are limited to; large values around x
    reach neither values nor scales, and nothing around q and the scales is written."""
    rows, cols, experts = 300, 136, len(off) - 1
    x = rows_of(rows, cols, DTYPES[name])
    room = torch.full((rows + 400, cols + 8), 3e4, dtype=x.dtype, device="cuda")
    room[200:500, :cols] = x.cuda()
    stored = (rows + 127 * min(rows, experts)) // 128 * 128
    values = torch.full((stored + 256, 144), 0x5A, dtype=torch.uint8, device="cuda")
    scales = torch.full((stored // 128 + 2, cols), 77.0, device="cuda")
    out = fp8.Quantized(values.view(E4M3)[128:128 + stored, :cols], scales[1:-1])
    offsets = torch.tensor([2 ** 30, *off, 2 ** 30], dtype=torch.int32, device="cuda")[1:-1]
    fp8.quantize(room[200:500, :cols], "columns", offsets=offsets, out=out)
    at = 0
    for b, e in limited(off, rows)[0]:
        if b < e:
            v, s = quantize64(x[b:e], "columns", E4M3)
            same(out.values[at:at + e - b], v)
            same(out.scales[at // 128:at // 128 + len(s)], s.astype(np.float64))
            assert not out.values[at + e - b:at + 128 * len(s)].view(torch.uint8).any()
            at += 128 * len(s)
    assert not out.values[at:].view(torch.uint8).any() and bool((out.scales[at // 128:] == 2.0 ** -126).all())
    out.values.view(torch.uint8).fill_(0x5A)
    assert bool((values == 0x5A).all()) and bool((scales[0] == 77).all() and (scales[-1] == 77).all())


def test_quantize_nothing(fp8):
    for shape in ((0, 64), (64, 0), (0, 0)):
        for block in ("rows", "columns", "blocks"):
            q = fp8.quantize(torch.empty(shape, device="cuda"), block)
            assert q.values.shape == shape
    off = torch.zeros(5, dtype=torch.int32, device="cuda")
    assert fp8.quantize(torch.empty((0, 64), device="cuda"), "columns", offsets=off).values.shape == (0, 64)


# ---------------------------------------------------------------------- products


def operands(fp8, rows, N, K, trans, ta=E4M3, tb=E4M3, experts=0, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + rows + 7 * N + 31 * K)
    x = torch.randn((rows, K), generator=g, device="cuda") * torch.exp(torch.randn((rows, 1), generator=g, device="cuda"))
    shape = (N, K) if trans else (K, N)
    w = torch.randn((experts, *shape) if experts else shape, generator=g, device="cuda")
    return fp8.quantize(x, "rows", dtype=ta), fp8.quantize(w, "blocks", dtype=tb)


def op(w, trans):
    return w.transpose(-1, -2) if trans else w


SIZES = [(1, 1, 1), (1, 256, 128), (3, 5, 16), (31, 33, 129), (128, 128, 128), (129, 257, 127), (255, 256, 384),
         (256, 512, 640), (257, 300, 1000), (600, 40, 260), (33, 700, 2049)]


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("rows,N,K", SIZES)
def test_gemm(fp8, rows, N, K, trans):
    a, b = operands(fp8, rows, N, K, trans)
    A, B = meaning(a, "rows"), op(meaning(b, "blocks"), trans)
    for dtype in DTYPES.values():
        check_product(fp8.gemm(a, b, transB=trans, dtype=dtype), A, B, K, f"{dtype}")


@pytest.mark.parametrize("rows", [1, 2, 8, 9, 16, 17, 32])
@pytest.mark.parametrize("N,K", [(1, 1), (15, 128), (17, 127), (129, 1040), (260, 1153), (40, 3201)])
def test_gemm_of_few_rows(fp8, rows, N, K):
    for ta, tb in ((E4M3, E4M3), (E5M2, E4M3), (E4M3, E5M2), (E5M2, E5M2)):
        a, b = operands(fp8, rows, N, K, True, ta, tb, seed=rows)
        A, B = meaning(a, "rows"), meaning(b, "blocks").t()
        for dtype in DTYPES.values():
            room = torch.full((rows + 1, N + 3), 7.0, dtype=dtype, device="cuda")
            check_product(fp8.gemm(a, b, out=room[:rows, :N], transB=True), A, B, K, f"{dtype}")
            assert bool((room[rows:] == 7).all() and (room[:, N:] == 7).all())


def test_gemm_of_few_rows_reads_no_padding(fp8):
    """Bytes behind the last column, whatever they are, and NaN in one row."""
    a, b = operands(fp8, 9, 50, 200, True)
    want = fp8.gemm(a, b, transB=True)
    wide = [torch.full((*t.shape[:-1], 208), 0x7F, dtype=torch.uint8, device="cuda") for t in (a.values, b.values)]
    for w, t in zip(wide, (a.values, b.values)):
        w[..., :200] = t.view(torch.uint8)
    aw, bw = (fp8.Quantized(w.view(E4M3)[..., :200], t.scales) for w, t in zip(wide, (a, b)))
    assert torch.equal(fp8.gemm(aw, bw, transB=True), want)
    wide[0][4, 130] = 0x7F
    got = fp8.gemm(aw, bw, transB=True)
    assert bool(got[4].isnan().all()) and torch.equal(got[:4], want[:4]) and torch.equal(got[5:], want[5:])


@pytest.mark.parametrize("ta", [E4M3, E5M2])
@pytest.mark.parametrize("tb", [E4M3, E5M2])
def test_gemm_types(fp8, ta, tb):
    for trans in (False, True):
        a, b = operands(fp8, 200, 300, 400, trans, ta, tb)
        check_product(fp8.gemm(a, b, transB=trans, dtype=torch.float32), meaning(a, "rows"),
                      op(meaning(b, "blocks"), trans), 400)
    x, y = (fp8.quantize(torch.randn((300, n), device="cuda"), "columns", dtype=t) for n, t in ((200, ta), (150, tb)))
    check_product(fp8.gemm_wgrad(x, y), meaning(x, "columns").t(), meaning(y, "columns"), 300)


GROUPS = [([40, 0, 256, 1, 300], 0), ([0, 0, 5], 9), ([128], 0), ([1] * 12, 3), ([257, 255], 1), ([0, 0], 4)]


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("counts,tail", GROUPS)
def test_gemm_of_groups(fp8, counts, tail, trans):
    rows, N, K, E = sum(counts) + tail, 270, 200, len(counts)
    a, b = operands(fp8, rows, N, K, trans, experts=E)
    off = offsets_of(counts).cuda()
    out = torch.full((rows, N), float("nan"), device="cuda")
    c = fp8.gemm(a, b, off, out, transB=trans)
    A, B, at = meaning(a, "rows"), op(meaning(b, "blocks"), trans), 0
    for e, n in enumerate(counts):
        if n:
            check_product(c[at:at + n], A[at:at + n], B[e], K, f"group {e}")
        at += n
    assert not c[at:].any() and bool(torch.isfinite(c).all())


@pytest.mark.parametrize("counts,tail", GROUPS)
@pytest.mark.parametrize("M,N", [(1, 1), (130, 270), (256, 96), (300, 33)])
def test_wgrad_of_groups(fp8, counts, tail, M, N):
    rows, E = sum(counts) + tail, len(counts)
    g = torch.Generator(device="cuda").manual_seed(rows + M)
    x, y = (torch.randn((rows, n), generator=g, device="cuda") for n in (M, N))
    off = offsets_of(counts).cuda()
    a, b = fp8.quantize(x, "columns", offsets=off), fp8.quantize(y, "columns", dtype=E5M2, offsets=off)
    out = torch.full((E, M, N), float("nan"), device="cuda")
    c = fp8.gemm_wgrad(a, b, off, out)
    A, B, at = meaning(a, "columns"), meaning(b, "columns"), 0
    for e, n in enumerate(counts):
        blocks = -(-n // 128)
        r = slice(128 * at, 128 * (at + blocks))
        check_product(c[e], A[r].t(), B[r], n, f"group {e}")
        at += blocks
    for dtype in (torch.bfloat16, torch.float16):
        half = fp8.gemm_wgrad(a, b, off, dtype=dtype)
        assert torch.equal(half, c.to(dtype))


@pytest.mark.parametrize("rows,M,N", [(1, 1, 1), (127, 64, 40), (128, 128, 128), (300, 257, 260), (1025, 33, 300)])
def test_wgrad(fp8, rows, M, N):
    g = torch.Generator(device="cuda").manual_seed(rows + M)
    a, b = (fp8.quantize(torch.randn((rows, n), generator=g, device="cuda"), "columns") for n in (M, N))
    check_product(fp8.gemm_wgrad(a, b), meaning(a, "columns").t(), meaning(b, "columns"), rows)


@pytest.mark.parametrize("counts,tail", [(None, 0), ([3000], 0), ([8000, 0, 130, 301], 5), ([3000, 2500, 900], 0)])
@pytest.mark.parametrize("M,N", [(1, 1), (130, 270), (64, 96)])
def test_wgrad_in_slices(fp8, counts, tail, M, N):
    """Few matrices over many rows, whose rows are summed in slices."""
    rows = 5003 if counts is None else sum(counts) + tail
    g = torch.Generator(device="cuda").manual_seed(rows + M)
    x, y = (torch.randn((rows, n), generator=g, device="cuda") for n in (M, N))
    off = None if counts is None else offsets_of(counts).cuda()
    a, b = fp8.quantize(x, "columns", offsets=off), fp8.quantize(y, "columns", dtype=E5M2, offsets=off)
    A, B = meaning(a, "columns"), meaning(b, "columns")
    for dtype in DTYPES.values():
        shape = (M, N) if counts is None else (len(counts), M, N)
        room = torch.full((*shape[:-2], M + 1, N + 3), 7.0, dtype=dtype, device="cuda")
        c = fp8.gemm_wgrad(a, b, off, room[..., :M, :N])
        assert bool((room[..., M:, :] == 7).all() and (room[..., N:] == 7).all())
        assert torch.equal(fp8.gemm_wgrad(a, b, off, dtype=dtype), c)
        at = 0
        for e, n in enumerate([rows] if counts is None else counts):
            end = at + -(-n // 128) * 128
            check_product(c if counts is None else c[e], A[at:end].t(), B[at:end], max(n, 1), f"{dtype} group {e}")
            at = end


@pytest.mark.parametrize("a,b", [(2.0 ** 100, 2.0 ** -100), (2.0 ** -100, 2.0 ** 100), (2.0 ** -126, 2.0 ** 120)])
def test_scales_far_from_one(fp8, a, b):
    """Two scales whose product is in range, where a block's sum times one of them would not be."""
    g = torch.Generator(device="cuda").manual_seed(17)

    def far(shape, block, dtype, size, experts=0):
        s = {"rows": (-(-shape[1] // 128), shape[0]), "columns": (-(-shape[0] // 128), shape[1]),
             "blocks": (-(-shape[0] // 128), -(-shape[1] // 128))}[block]
        lead = (experts,) if experts else ()
        q = fp8.quantize(torch.randn((*lead, *shape), generator=g, device="cuda"), block, dtype=dtype)
        return fp8.Quantized(q.values, size * (1 + torch.rand((*lead, *s), generator=g, device="cuda") / 2))

    for ta, tb in ((E4M3, E4M3), (E5M2, E5M2), (E5M2, E4M3)):
        for rows, trans in ((8, True), (300, True), (300, False)):
            x, w = far((rows, 700), "rows", ta, a), far((260, 700) if trans else (700, 260), "blocks", tb, b)
            check_product(fp8.gemm(x, w, transB=trans, dtype=torch.float32), meaning(x, "rows"),
                          op(meaning(w, "blocks"), trans), 700, f"rows {rows} {trans}")
        off = torch.tensor([0, 100, 384], dtype=torch.int32, device="cuda")
        x, w = far((384, 200), "rows", ta, a), far((140, 200), "blocks", tb, b, 2)
        c = fp8.gemm(x, w, off, transB=True, dtype=torch.float32)
        for e, r in enumerate((slice(0, 100), slice(100, 384))):
            check_product(c[r], meaning(x, "rows")[r], meaning(w, "blocks")[e].t(), 200, f"group {e}")
        for rows, M, N in ((300, 130, 270), (5003, 130, 270)):  # the second in slices
            x, y = far((rows, M), "columns", ta, a), far((rows, N), "columns", tb, b)
            check_product(fp8.gemm_wgrad(x, y), meaning(x, "columns").t(), meaning(y, "columns"), rows, f"wgrad {rows}")


def near(got, a, b, terms, what):
    """check_product on the GPU, for large results."""
    exact, size = a @ b, a.abs() @ b.abs()
    limit = 2 * (terms + 1) * 2.0 ** -23 * size + ROUNDING[got.dtype] * exact.abs() + TINY[got.dtype]
    bad = ~((got.double() - exact).abs() <= limit)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} out of bound"


@pytest.mark.parametrize("name", list(DTYPES))
@pytest.mark.parametrize("trans", [False, True])
def test_gemm_many_tiles(fp8, name, trans):
    """More tiles than SM pairs, so that a pair takes several: dense, and in groups with ends of any size."""
    a, b = operands(fp8, 4100, 4200, 260, trans)
    out = torch.full((4100, 4200), float("nan"), dtype=DTYPES[name], device="cuda")
    near(fp8.gemm(a, b, out=out, transB=trans), meaning(a, "rows"), op(meaning(b, "blocks"), trans), 260, "dense")
    counts = [270, 0, 5, 256, 300, 700, 31, 128] * 5
    rows = sum(counts) + 300
    a, b = operands(fp8, rows, 600, 390, trans, experts=len(counts))
    out = torch.full((rows, 600), float("nan"), dtype=DTYPES[name], device="cuda")
    fp8.gemm(a, b, offsets_of(counts).cuda(), out, transB=trans)
    A, B, at = meaning(a, "rows"), op(meaning(b, "blocks"), trans), 0
    for e, n in enumerate(counts):
        near(out[at:at + n], A[at:at + n], B[e], 390, f"group {e}")
        at += n
    assert not out[at:].any()


@pytest.mark.parametrize("name", list(DTYPES))
def test_wgrad_many_tiles(fp8, name):
    g = torch.Generator(device="cuda").manual_seed(8)
    x, y = (torch.randn((1100, n), generator=g, device="cuda") for n in (2600, 2500))
    a, b = fp8.quantize(x, "columns"), fp8.quantize(y, "columns", dtype=E5M2)
    out = torch.full((2600, 2500), float("nan"), dtype=DTYPES[name], device="cuda")
    near(fp8.gemm_wgrad(a, b, out=out), meaning(a, "columns").t(), meaning(b, "columns"), 1100, "dense")
    counts = [270, 0, 5, 256, 300, 1700, 31, 128] * 5
    off = offsets_of(counts).cuda()
    x, y = (torch.randn((sum(counts) + 50, n), generator=g, device="cuda") for n in (300, 500))
    a, b = fp8.quantize(x, "columns", offsets=off), fp8.quantize(y, "columns", dtype=E5M2, offsets=off)
    out = torch.full((len(counts), 300, 500), float("nan"), dtype=DTYPES[name], device="cuda")
    fp8.gemm_wgrad(a, b, off, out)
    A, B, at = meaning(a, "columns"), meaning(b, "columns"), 0
    for e, n in enumerate(counts):
        end = at + -(-n // 128) * 128
        near(out[e], A[at:end].t(), B[at:end], n, f"matrix {e}")
        at = end


def test_a_row_depends_on_itself(fp8):
    """The same row gives the same bits among others and in a group, and, where few rows have a kernel of their own,
    the same bits among few."""
    a, b = operands(fp8, 700, 520, 2000, True)

    def some(r):
        return fp8.gemm(fp8.Quantized(a.values[r], a.scales[:, r].contiguous()), b, transB=True, dtype=torch.float32)

    all_rows = fp8.gemm(a, b, transB=True, dtype=torch.float32)
    for r in (slice(3, 50), slice(255, 600)):
        assert torch.equal(some(r), all_rows[r])
    few = some(slice(40, 72))
    for n in (1, 8, 9, 16, 17):
        assert torch.equal(some(slice(40, 40 + n)), few[:n])
    stack = fp8.Quantized(b.values[None].repeat(3, 1, 1), b.scales[None].repeat(3, 1, 1))
    off = torch.tensor([0, 37, 37, 700], dtype=torch.int32, device="cuda")
    assert torch.equal(fp8.gemm(a, stack, off, transB=True, dtype=torch.float32), all_rows)


@pytest.mark.parametrize("pad,offset", [(0, 0), (1, 0), (3, 1), (8, 8)])
def test_strides_and_what_lies_around(fp8, pad, offset):
    a, b = operands(fp8, 300, 260, 300, True)
    for dtype in DTYPES.values():
        want = fp8.gemm(a, b, transB=True, dtype=dtype)
        out = strided(torch.zeros((300, 260), dtype=dtype), pad, offset)
        assert torch.equal(fp8.gemm(a, b, out=out, transB=True), want)
        assert canaries_intact(out)
    x, y = (fp8.quantize(torch.randn((300, n), device="cuda"), "columns") for n in (140, 150))
    want = fp8.gemm_wgrad(x, y)
    out = strided(torch.zeros((140, 150)), pad, offset)
    assert torch.equal(fp8.gemm_wgrad(x, y, out=out), want) and canaries_intact(out)
    # Operands with rows further apart, and matrices of a stack further apart than they are long.
    wide = torch.zeros((300, 512), dtype=torch.uint8, device="cuda").view(E4M3)
    wide.view(torch.uint8)[:, 16:316] = a.values.view(torch.uint8)
    stack = torch.zeros((2, 400, 320), dtype=torch.uint8, device="cuda").view(E4M3)
    stack.view(torch.uint8)[:, :260, :300] = b.values.view(torch.uint8)
    b2 = fp8.Quantized(stack[:, :260, :300], b.scales[None].repeat(2, 1, 1))
    off = torch.tensor([0, 100, 300], dtype=torch.int32, device="cuda")
    got = fp8.gemm(fp8.Quantized(wide[:, 16:316], a.scales), b2, off, transB=True)
    assert torch.equal(got, fp8.gemm(a, b, transB=True))


def test_nan_stays_in_its_row(fp8):
    x = torch.randn((300, 260), device="cuda")
    x[7, 200], x[290, 0] = float("nan"), float("inf")
    w = torch.randn((300, 260), device="cuda")
    clean = x.clone()
    clean[7, 200] = clean[290, 0] = 0
    b = fp8.quantize(w, "blocks")
    bad = fp8.gemm(fp8.quantize(x, "rows"), b, transB=True)
    assert bool(torch.isnan(bad[[7, 290]]).all())
    rest = [r for r in range(300) if r not in (7, 290)]
    assert torch.equal(bad[rest], fp8.gemm(fp8.quantize(clean, "rows"), b, transB=True)[rest])
    # A group's NaN does not reach the next group, whose rows share its tiles' loads.
    off = torch.tensor([0, 8, 300], dtype=torch.int32, device="cuda")
    stack = fp8.quantize(torch.stack([w, w]), "blocks")
    assert bool(torch.isfinite(fp8.gemm(fp8.quantize(x, "rows"), stack, off, transB=True)[rest]).all())
    g = fp8.gemm_wgrad(fp8.quantize(x, "columns", offsets=off), fp8.quantize(x, "columns", offsets=off), off)
    assert bool(torch.isnan(g[0, 200]).all()) and bool(torch.isnan(g[1, 0]).all())
    assert bool(torch.isfinite(g[0, :200, :200]).all()) and bool(torch.isfinite(g[1, 1:, 1:]).all())


def test_products_of_nothing(fp8):
    q = lambda r, c, block: fp8.quantize(torch.zeros((r, c), device="cuda"), block)  # noqa: E731
    assert fp8.gemm(q(0, 64, "rows"), q(32, 64, "blocks"), transB=True).shape == (0, 32)
    assert fp8.gemm(q(4, 64, "rows"), q(0, 64, "blocks"), transB=True).shape == (4, 0)
    out = torch.full((4, 32), 5.0, device="cuda")
    fp8.gemm(q(4, 0, "rows"), q(32, 0, "blocks"), out=out, transB=True)
    assert not out.any()
    out = torch.full((2, 16, 32), 5.0, device="cuda")
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    fp8.gemm_wgrad(q(0, 16, "columns"), q(0, 32, "columns"), off, out)
    assert not out.any()


def test_products_of_nothing_into_rows_far_apart(fp8):
    """A sum of nothing is zero in rows more than 2^31 bytes apart, too."""
    q = lambda r, c, block: fp8.quantize(torch.zeros((r, c), device="cuda"), block)  # noqa: E731
    pitch = 2 ** 29 + 16
    store = torch.full((2 * pitch,), 5.0, device="cuda")
    out = store.as_strided((2, 32), (pitch, 1))
    fp8.gemm(q(2, 0, "rows"), q(32, 0, "blocks"), out=out, transB=True)
    assert not out.any() and bool((store[32:64] == 5).all()) and bool((store[pitch + 32:] == 5).all())
    out.fill_(5.0)
    fp8.gemm_wgrad(q(0, 2, "columns"), q(0, 32, "columns"), out=out)
    assert not out.any()


def test_elements_past_32_bits(fp8):
    """Operands and results of more than 2^31 elements: their last rows and columns."""
    rows, wide, last = 270000, 8192, 300
    x = torch.empty((rows, wide), dtype=torch.bfloat16, device="cuda")
    assert x.numel() > 2 ** 31
    x.normal_(generator=torch.Generator(device="cuda").manual_seed(4))
    by_row, by_column = fp8.quantize(x, "rows"), fp8.quantize(x, "columns")
    assert torch.equal(fp8.quantize(x, "blocks").scales[-3:], fp8.quantize(x[rows // 128 * 128 - 256:], "blocks").scales)
    end = fp8.quantize(x[-last:], "rows")
    assert torch.equal(by_row.values[-last:].view(torch.uint8), end.values.view(torch.uint8))
    assert torch.equal(by_row.scales[:, -last:], end.scales)
    whole = rows // 128 * 128 - 256
    values, scales = reference8(x[whole:], "columns", E4M3)
    assert torch.equal(by_column.values[whole:].view(torch.uint8), values)
    assert torch.equal(by_column.scales[whole // 128:], scales)
    w = fp8.quantize(torch.randn((128, wide), device="cuda"), "blocks")
    assert torch.equal(fp8.gemm(by_row, w, transB=True)[-last:], fp8.gemm(end, w, transB=True))
    # A result of as many, from a short sum.
    short = fp8.Quantized(by_row.values[:, :128], by_row.scales[:1].contiguous())
    of_end = fp8.Quantized(end.values[:, :128], end.scales[:1].contiguous())
    w = fp8.quantize(torch.randn((wide, 128), device="cuda"), "blocks")
    for dtype in (torch.float32, torch.bfloat16):
        assert torch.equal(fp8.gemm(short, w, transB=True, dtype=dtype)[-last:], fp8.gemm(of_end, w, transB=True, dtype=dtype))
    # The gradient's sum over all rows, of which only the last ones are not zero.
    y = torch.zeros((rows, 64), device="cuda")
    y[-last:] = torch.randn((last, 64), device="cuda")
    dy = fp8.quantize(y, "columns")
    near(fp8.gemm_wgrad(by_column, dy), meaning(fp8.Quantized(by_column.values[whole:], by_column.scales[whole // 128:]),
                                                "columns").t(),
         meaning(fp8.Quantized(dy.values[whole:], dy.scales[whole // 128:]), "columns"), rows - whole, "gradient")


def test_offsets_are_limited(fp8):
    a, b = operands(fp8, 200, 64, 128, True, experts=2)
    for off in ([0, 1000, 2000], [0, 150, 100], [0, -3, 200]):
        t = torch.tensor(off, dtype=torch.int32, device="cuda")
        assert bool(torch.isfinite(fp8.gemm(a, b, t, transB=True)).all())
        x = fp8.quantize(torch.randn((200, 64), device="cuda"), "columns", offsets=t)
        assert bool(torch.isfinite(fp8.gemm_wgrad(x, x, t)).all())


@pytest.mark.parametrize("off", BAD_OFFSETS, ids=str)
def test_products_of_limited_offsets(fp8, off):
    """Products of the groups that offsets are limited to, into outputs that hold NaN. Rows that decreasing bounds give
    to two groups may hold either's."""
    rows, N, K, E = 300, 200, 140, len(off) - 1
    t = torch.tensor(off, dtype=torch.int32, device="cuda")
    groups, behind = limited(off, rows)
    for trans in (False, True):
        a, b = operands(fp8, rows, N, K, trans, experts=E)
        room = torch.full((rows + 64, N), float("nan"), device="cuda")
        c = fp8.gemm(a, b, t, room[32:-32], transB=trans)
        A, B = meaning(a, "rows"), op(meaning(b, "blocks"), trans)
        of = [[e for e, (x, y) in enumerate(groups) if x <= r < y] + ([E] if r >= behind else []) for r in range(rows)]
        for r in range(rows):
            if len(of[r]) == 1:
                check_product(c[r:r + 1], A[r:r + 1], B[of[r][0]] if of[r][0] < E else torch.zeros_like(B[0]), K, f"{r}")
        assert all(of) and bool(torch.isfinite(c).all())
        assert bool(room[:32].isnan().all() and room[-32:].isnan().all())
    g = torch.Generator(device="cuda").manual_seed(rows)
    x, y = (fp8.quantize(torch.randn((rows, n), generator=g, device="cuda"), "columns", offsets=t) for n in (130, 70))
    room = torch.full((E + 2, 130, 70), float("nan"), device="cuda")
    c = fp8.gemm_wgrad(x, y, t, room[1:-1])
    X, Y, at = meaning(x, "columns"), meaning(y, "columns"), 0
    for e, (b, end) in enumerate(groups):
        blocks = -(-(end - b) // 128)
        r = slice(128 * at, 128 * (at + blocks))
        check_product(c[e], X[r].t(), Y[r], end - b, f"matrix {e}")
        at += blocks
    assert bool(room[0].isnan().all() and room[-1].isnan().all())


def test_gradients_against_differences(fp8):
    """The products are bilinear: with changes E and G of the values (8-bit ones, at the same scales), <D, (A + E) B -
    A B> = <D B^T, E> and <D, A (B + G) - A B> = <A^T D, G>."""
    g = torch.Generator(device="cuda").manual_seed(3)
    S, N, K = 256, 128, 256

    def pick(*shape):  # whole numbers: sums below 2^24 are exact
        return torch.randint(-4, 5, shape, generator=g, device="cuda").float()

    def quantized(v, block):
        high, wide = {"rows": (1, 128), "columns": (128, 1), "blocks": (128, 128)}[block]
        s = torch.ones((-(-v.shape[0] // high), -(-v.shape[1] // wide)), device="cuda")
        return fp8.Quantized(v.to(E4M3), s.t().contiguous() if block == "rows" else s)

    A, B, D, E, G = pick(S, K), pick(K, N), pick(S, N), pick(S, K), pick(K, N)
    f = lambda a, b: fp8.gemm(quantized(a, "rows"), quantized(b, "blocks"), dtype=torch.float32).double()  # noqa: E731
    dA = fp8.gemm(quantized(D, "rows"), quantized(B, "blocks"), transB=True, dtype=torch.float32).double()
    dB = fp8.gemm_wgrad(quantized(A, "columns"), quantized(D, "columns")).double()
    assert float((D * (f(A + E, B) - f(A, B))).sum()) == float((dA * E).sum())
    assert float((D * (f(A, B + G) - f(A, B))).sum()) == float((dB * G).sum())


def test_refusals(fp8):
    a, b = operands(fp8, 32, 64, 128, True)
    with pytest.raises(ValueError, match="16-byte"):
        fp8.gemm(fp8.Quantized(a.values[:, 1:], a.scales), fp8.Quantized(b.values[:, 1:], b.scales), transB=True)
    with pytest.raises(ValueError, match="inner"):
        fp8.gemm(a, b)
    with pytest.raises(ValueError, match="shape"):
        fp8.gemm(fp8.Quantized(a.values, a.scales.t().contiguous()), b, transB=True)
    with pytest.raises(ValueError, match="whole blocks"):
        x = fp8.quantize(torch.zeros((130, 64), device="cuda"), "columns")
        fp8.gemm_wgrad(x, x, torch.zeros(3, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        fp8.quantize(torch.zeros((4, 4), device="cuda"), "rows", offsets=torch.zeros(3, dtype=torch.int32, device="cuda"))
    with pytest.raises(TypeError):
        fp8.gemm(a, b, transB=True, dtype=torch.float64)

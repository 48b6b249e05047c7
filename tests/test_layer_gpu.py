"""The mixture-of-experts layer for a few tokens against its definition in 64 bits."""

import numpy as np
import pytest
import torch

from tests.experts_harness import DTYPES, canaries_intact, random_ids, strided
from tests.fp8_harness import E4M3, E5M2, check_layer, meaning

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def layer():
    from dense_fp32_matrix_major_gb300 import layer

    return layer


@pytest.fixture(scope="module")
def fp8():
    from dense_fp32_matrix_major_gb300 import fp8

    return fp8


def case(tokens, top_k, experts, width, hidden, dtype, gated, drop=0.0, skew=0.0, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + tokens + 3 * width + 5 * hidden)

    def randn(*shape, scale=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)

    ids = random_ids(np.random.default_rng(seed + tokens), tokens, top_k, experts, drop, skew).cuda()
    return {"x": randn(tokens, width), "ids": ids, "weights": torch.rand((tokens, top_k), generator=g, device="cuda"),
            "w1": randn(experts, hidden * (2 if gated else 1), width, scale=max(width, 1) ** -0.5),
            "w2": randn(experts, width, hidden, scale=max(hidden, 1) ** -0.5)}


def check(layer, c, gated, act, fp8=None, to=None, what=""):
    w1, w2 = c["w1"], c["w2"]
    if fp8 is not None:
        w1, w2 = fp8.quantize(w1, "blocks", dtype=to), fp8.quantize(w2, "blocks", dtype=to)
        d1, d2 = meaning(w1, "blocks"), meaning(w2, "blocks")
    else:
        d1, d2 = w1.double(), w2.double()
    y = layer.forward(c["x"], c["ids"], c["weights"], w1, w2, gated=gated, activation=act)
    check_layer(y, c["x"], c["ids"], c["weights"], d1, d2, gated, act, what)
    return y


# tokens, top_k, experts, width, hidden
SIZES = [(1, 1, 1, 1, 1), (1, 8, 64, 256, 64), (2, 2, 4, 64, 1), (3, 4, 9, 301, 133), (1, 1, 3, 8, 2000),
         (5, 2, 3, 1000, 72), (17, 1, 1, 130, 96), (9, 6, 5, 520, 248), (40, 4, 6, 328, 160), (64, 8, 8, 256, 512),
         (512, 1, 40, 64, 40), (8, 64, 100, 72, 24), (4, 2, 4096, 32, 16), (2, 2, 2, 5000, 24)]


@pytest.mark.parametrize("name", list(DTYPES))
@pytest.mark.parametrize("size", SIZES, ids=["x".join(map(str, s)) for s in SIZES])
def test_layer(layer, name, size):
    for gated, act in ((True, "silu"), (False, "gelu")):
        check(layer, case(*size, DTYPES[name], gated, drop=0.1), gated, act, what=f"{gated}")


@pytest.mark.parametrize("name", list(DTYPES))
@pytest.mark.parametrize("to", [E4M3, E5M2])
@pytest.mark.parametrize("size", SIZES[:12], ids=["x".join(map(str, s)) for s in SIZES[:12]])
def test_layer_of_8_bit_matrices(layer, fp8, name, to, size):
    for gated, act in ((True, "silu"), (False, "relu")):
        check(layer, case(*size, DTYPES[name], gated, drop=0.1), gated, act, fp8, to, f"{gated}")


@pytest.mark.parametrize("act", ["silu", "gelu", "relu", None])
@pytest.mark.parametrize("gated", [False, True])
def test_activations(layer, act, gated):
    for dtype in DTYPES.values():
        check(layer, case(6, 2, 4, 128, 96, dtype, gated), gated, act)


@pytest.mark.parametrize("name", list(DTYPES))
def test_all_pairs_of_one_expert(layer, name):
    """Entries of eight pairs each, the last of any number; the same expert twice for a token."""
    for tokens in (1, 7, 8, 9, 16, 33, 64):
        c = case(tokens, 2, 3, 136, 72, DTYPES[name], True)
        c["ids"][:] = 1
        check(layer, c, True, "silu", what=str(tokens))


def test_dropped_pairs(layer):
    for dtype in DTYPES.values():
        c = case(6, 3, 4, 96, 80, dtype, True)
        c["ids"][0] = torch.tensor([-1, 4, 1 << 40])
        c["ids"][1, 1] = -7
        c["weights"][0] = float("nan")
        c["weights"][1, 1] = float("inf")
        y = check(layer, c, True, "silu")
        assert not y[0].any()
        c["ids"][:] = -1
        assert not layer.forward(c["x"], c["ids"], c["weights"], c["w1"], c["w2"], gated=True).any()
        c["ids"] = torch.randint(-1, 4, (6, 3), device="cuda", dtype=torch.int32)
        c["weights"] = torch.rand((6, 3), device="cuda")
        check(layer, c, True, "silu")


@pytest.mark.parametrize("pad,offset", [(0, 0), (1, 0), (0, 1), (8, 8), (3, 5)])
@pytest.mark.parametrize("name", list(DTYPES))
def test_strides(layer, name, pad, offset):
    dtype = DTYPES[name]
    c = case(5, 2, 3, 136, 72, dtype, True)
    want = layer.forward(c["x"], c["ids"], c["weights"], c["w1"], c["w2"], gated=True)
    flat = {k: strided(c[k].flatten(0, -2), pad, offset) for k in ("x", "w1", "w2")}
    out = strided(torch.zeros((5, 136), dtype=dtype), pad, offset)
    args = {k: (v if k == "x" else v.as_strided(c[k].shape, (v.stride(0) * c[k].shape[1], v.stride(0), 1),
                                                v.storage_offset())) for k, v in flat.items()}
    y = layer.forward(args["x"], c["ids"], c["weights"], args["w1"], args["w2"], gated=True, out=out)
    check_layer(y, c["x"], c["ids"], c["weights"], c["w1"].double(), c["w2"].double(), True, "silu")
    assert canaries_intact(out)
    if pad == offset == 0:
        assert torch.equal(y, want)


def among_nan(t, pitch, offset):
    """t's values in rows of `pitch` from value `offset` of a buffer on, NaN (0x7F in 8 bits) everywhere else."""
    rows = t.flatten(0, -2)
    bits = t.element_size() == 1
    room = torch.full((offset + rows.shape[0] * pitch + 64,), 0x7F if bits else float("nan"),
                      dtype=torch.uint8 if bits else t.dtype, device="cuda")
    strides = (t.shape[-2] * pitch, pitch, 1)[-t.dim():]
    view = room.as_strided(t.shape, strides, offset)
    view.copy_(t.view(torch.uint8) if bits else t)
    return view.view(t.dtype) if bits else view


@pytest.mark.parametrize("name", list(DTYPES))
@pytest.mark.parametrize("width,hidden", [(133, 71), (8, 3), (1, 1), (520, 261), (300, 640)])
def test_what_lies_around_rows_is_not_read_as_values(layer, fp8, name, width, hidden):
    """Rows on 16-byte boundaries that end anywhere, and rows anywhere, with NaN before, between and behind them."""
    dtype = DTYPES[name]
    for gated in (False, True):
        c = case(9, 2, 3, width, hidden, dtype, gated, drop=0.1)
        d1, d2 = c["w1"].double(), c["w2"].double()
        for p1, p2, px, o in ((-(-width // 8) * 8, -(-hidden // 8) * 8 + 8, -(-width // 8) * 8, 0), (width, hidden, width, 5), (width + 3, hidden + 1, width + 5, 1),
                              (width + 7, hidden + 2, -(-width // 8) * 8, 8)):
            y = layer.forward(among_nan(c["x"], px, o), c["ids"], c["weights"], among_nan(c["w1"], p1, o),
                              among_nan(c["w2"], p2, o), gated=gated, activation="gelu")
            check_layer(y, c["x"], c["ids"], c["weights"], d1, d2, gated, "gelu", f"{gated} {p1} {p2} {px} {o}")
        q1, q2 = fp8.quantize(c["w1"], "blocks"), fp8.quantize(c["w2"], "blocks")
        e1, e2 = meaning(q1, "blocks"), meaning(q2, "blocks")
        w1, w2 = (fp8.Quantized(among_nan(q.values, -(-q.values.shape[-1] // 16) * 16 + 16, 32), q.scales) for q in (q1, q2))
        for px, o in ((width, 0), (width + 1, 3), (-(-width // 8) * 8, 8)):
            y = layer.forward(among_nan(c["x"], px, o), c["ids"], c["weights"], w1, w2, gated=gated, activation="gelu")
            check_layer(y, c["x"], c["ids"], c["weights"], e1, e2, gated, "gelu", f"8 bits {gated} {px} {o}")


@pytest.mark.parametrize("name", list(DTYPES))
def test_infinities_and_nan(layer, fp8, name):
    """What is not finite stays with its token, and infinities are what IEEE arithmetic makes of them."""
    c = case(6, 2, 4, 128, 64, DTYPES[name], False)
    bad = dict(c, x=c["x"].clone())
    bad["x"][1, 5] = float("nan")
    bad["x"][4, 100] = float("inf")
    for w1, w2 in ((c["w1"], c["w2"]), tuple(fp8.quantize(c[w], "blocks") for w in ("w1", "w2"))):
        fine = layer.forward(c["x"], c["ids"], c["weights"], w1, w2, activation="relu")
        y = layer.forward(bad["x"], c["ids"], c["weights"], w1, w2, activation="relu")
        assert bool(torch.isnan(y[1]).all()) and not bool(torch.isfinite(y[4]).any())
        rest = [0, 2, 3, 5]
        assert torch.equal(y[rest], fine[rest])
    # Positive weights: an infinity in x is one in h and in y, not a NaN.
    y = layer.forward(bad["x"], c["ids"], c["weights"], torch.ones_like(c["w1"]), torch.ones_like(c["w2"]),
                      activation="relu")
    assert bool((y[4] == float("inf")).all()) and bool(torch.isfinite(y[rest]).all())


@pytest.mark.parametrize("name", list(DTYPES))
@pytest.mark.parametrize("held", ["same", "e5m2"])
def test_infinite_matrix_elements(layer, fp8, name, held):
    """An infinity in W1 or W2, times positive values: infinities of its sign where its expert is used, for a 16-bit W2
    perhaps NaN, and nothing elsewhere."""
    dtype = DTYPES[name]
    c = case(6, 2, 4, 136, 72, dtype, False)
    c["ids"] = torch.tensor([[0, 1], [1, 2], [2, 0], [3, 3], [0, 0], [-1, 1]], dtype=torch.int32, device="cuda")
    x, w1, w2 = (c[k].abs() + 0.125 for k in ("x", "w1", "w2"))
    run = lambda a, b: layer.forward(x, c["ids"], c["weights"] + 0.5, a, b, activation="relu")  # noqa: E731

    def matrices(w, at=None, sign=1):
        w = w.clone() if held == "same" else fp8.quantize(w, "blocks", dtype=E5M2)
        if at is not None and held == "same":
            w[at] = sign * float("inf")
        elif at is not None:
            w.values.view(torch.uint8)[at] = 0x7C if sign > 0 else 0xFC
        return w

    fine = run(matrices(w1), matrices(w2))
    assert bool(torch.isfinite(fine).all())
    has, rest = [0, 1, 5], [2, 3, 4]  # tokens of expert 1
    y = run(matrices(w1, (1, 30, 100)), matrices(w2))
    assert bool((y[has] == float("inf")).all()) and torch.equal(y[rest], fine[rest])
    y = run(matrices(w1), matrices(w2, (1, 90, 40), -1))
    assert torch.equal(y[rest], fine[rest])
    other = torch.arange(136, device="cuda") != 90
    assert torch.equal(y[:, other], fine[:, other])
    if held == "same" and dtype != torch.float32:
        assert not bool(torch.isfinite(y[has, 90]).any()) and not bool((y[has, 90] == float("inf")).any())
    else:
        assert bool((y[has, 90] == -float("inf")).all())


def test_outliers_at_zero_weights(layer, fp8):
    """A value of x far above the rest, at weights that are zero, costs the rest no digits."""
    for dtype in DTYPES.values():
        c = case(4, 2, 3, 256, 64, dtype, True)
        big = 6e4 if dtype == torch.float16 else 1e30
        c["w1"][:, :, 17] = 0
        want = layer.forward(c["x"], c["ids"], c["weights"], c["w1"], c["w2"], gated=True)
        q1, q2 = fp8.quantize(c["w1"], "blocks"), fp8.quantize(c["w2"], "blocks")
        want8 = layer.forward(c["x"], c["ids"], c["weights"], q1, q2, gated=True)
        c["x"][:, 17] = big
        assert torch.equal(layer.forward(c["x"], c["ids"], c["weights"], c["w1"], c["w2"], gated=True), want)
        assert torch.equal(layer.forward(c["x"], c["ids"], c["weights"], q1, q2, gated=True), want8)


def test_hidden_values_past_fp16(layer):
    """h above fp16's largest number, where y is within its range."""
    c = case(3, 2, 3, 64, 40, torch.float16, True)
    c["w1"] *= 300
    c["w2"] *= 1e-3
    check(layer, c, True, None)


def test_hidden_values_past_bf16(layer):
    """h between bf16's largest number and fp32's, which is finite in both."""
    x = torch.ones((1, 8), dtype=torch.bfloat16, device="cuda")
    w1, w2 = torch.zeros((1, 8, 8), device="cuda"), torch.zeros((1, 8, 8), device="cuda")
    w1[0, :, 0], w1[0, :, 1] = torch.finfo(torch.bfloat16).max, 1.2e36
    w1[0, 4:] *= -1
    w2[0] = 2.0 ** -100
    w2[0, :, 4:] *= -1
    one = torch.ones((1, 1), device="cuda")
    ids = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    h = x.double() @ w1[0].bfloat16().double().t()
    assert float(h.abs().max()) > torch.finfo(torch.bfloat16).max
    y = layer.forward(x, ids, one, w1.bfloat16(), w2.bfloat16(), activation=None)
    check_layer(y, x, ids, one, w1.bfloat16().double(), w2.bfloat16().double(), False, None)


@pytest.mark.parametrize("to", [E4M3, E5M2])
@pytest.mark.parametrize("name", list(DTYPES))
def test_8_bit_sums_that_overflow_before_their_scale(layer, fp8, name, to):
    """x or h so large that a block's values times it leave fp32, where scaled ones do not; a pair of an expert or more
    than an entry has, sums that one warp has and that several share, more columns of y than a block makes at once, and
    a NaN in another token."""
    dtype = DTYPES[name]
    for tokens, width, hidden in ((2, 300, 260), (20, 140, 130), (3, 2000, 2100), (2, 6000, 130)):
        for gated in (False, True):
            c = case(tokens, 2, 3, width, hidden, torch.float32, False)
            gate = [torch.full_like(c["w1"], width ** -0.5)] if gated else []  # the second half: near one

            def w1(first, second):
                return torch.cat([c["w1"] * 2.0 ** first, *(w * 2.0 ** second for w in gate)], 1)

            x = c["x"].to(dtype)
            jobs = [(x, w1(117, 0), c["w2"] * 2.0 ** -114)]  # h
            if dtype != torch.float16:
                jobs.append((x * 2.0 ** 122, w1(-64, -64) if gated else w1(-30, 0), c["w2"]))  # x
            for t, u1, u2 in jobs:
                q1, q2 = fp8.quantize(u1, "blocks", dtype=to), fp8.quantize(u2, "blocks", dtype=to)
                d1, d2 = meaning(q1, "blocks"), meaning(q2, "blocks")
                y = layer.forward(t, c["ids"], c["weights"], q1, q2, gated=gated, activation=None)
                assert bool(torch.isfinite(y).all())
                check_layer(y, t, c["ids"], c["weights"], d1, d2, gated, None, f"{tokens} {gated}")
                bad = t.clone()
                bad[1, 7] = float("nan")
                z = layer.forward(bad, c["ids"], c["weights"], q1, q2, gated=gated, activation=None)
                rest = [i for i in range(tokens) if i != 1]
                assert bool(z[1].isnan().all()) and torch.equal(z[rest], y[rest])


@pytest.mark.parametrize("name", ["bf16", "f16"])
def test_small_terms_beside_a_large_sum(layer, name):
    """A running sum of 2^24 that the last term takes back, with terms between whose sum over an instruction's 16 values
    is half of the sum's last place: what an instruction cuts off is lost for the slice of 128 that holds a large
    term, and not for the whole row. Enough features that a warp has whole rows of W1."""
    dtype, width, hidden = DTYPES[name], 16384, 16 * 16 * torch.cuda.get_device_properties(0).multi_processor_count
    row = torch.full((width,), 0.25)
    row[0] = row[-1] = 2.0 ** 12
    x = row.to(dtype).cuda()[None]
    row[-1] *= -1
    w1 = row.to(dtype).cuda().expand(1, hidden, width).contiguous()
    w2 = torch.zeros((1, width, hidden), dtype=dtype, device="cuda")
    w2[0].fill_diagonal_(1)
    y = layer.forward(x, torch.zeros((1, 1), dtype=torch.int32, device="cuda"), torch.ones((1, 1), device="cuda"), w1, w2,
                      activation=None)
    exact = (width - 2) / 16
    # Two slices with a large term: 65 additions of a chain, each off by 2^-23 of 2^24; 128 slices added, half a last
    # place of 2^24 each. Then y's rounding.
    limit = 2 * 65 * 2 + 128
    assert limit < exact / 2
    assert float((y.double() - exact).abs().max()) <= limit + 2.0 ** -8 * 2 * exact


def test_nothing(layer):
    f = lambda t, k, w, h: layer.forward(  # noqa: E731
        torch.zeros((t, w), device="cuda"), torch.zeros((t, k), dtype=torch.int64, device="cuda"),
        torch.ones((t, k), device="cuda"), torch.zeros((2, h, w), device="cuda"), torch.zeros((2, w, h), device="cuda"))
    assert f(0, 2, 16, 8).shape == (0, 16)
    assert f(3, 2, 0, 8).shape == (3, 0)
    out = torch.full((3, 16), 7.0, device="cuda")
    layer.forward(torch.zeros((3, 16), device="cuda"), torch.zeros((3, 2), dtype=torch.int64, device="cuda"),
                  torch.ones((3, 2), device="cuda"), torch.zeros((2, 0, 16), device="cuda"),
                  torch.zeros((2, 16, 0), device="cuda"), out=out)
    assert not out.any()


def test_same_bits_again(layer):
    for dtype in DTYPES.values():
        c = case(30, 4, 7, 520, 264, dtype, True)
        one = layer.forward(c["x"], c["ids"], c["weights"], c["w1"], c["w2"], gated=True)
        for _ in range(5):
            assert torch.equal(layer.forward(c["x"], c["ids"], c["weights"], c["w1"], c["w2"], gated=True), one)


def test_offsets_past_32_bits(layer):
    """Matrices whose elements lie more than 2^31 elements into the stack."""
    E, D, F = 1100, 1024, 2048
    w1 = torch.empty((E, F, D), dtype=torch.bfloat16, device="cuda").fill_(float("nan"))
    w2 = torch.empty((E, D, F), dtype=torch.bfloat16, device="cuda").fill_(float("nan"))
    assert w1.numel() > 2 ** 31
    used = [0, 1099, 1050]
    for e in used:
        w1[e] = torch.randn((F, D), device="cuda") * D ** -0.5
        w2[e] = torch.randn((D, F), device="cuda") * F ** -0.5
    x = torch.randn((2, D), device="cuda").bfloat16()
    ids = torch.tensor([[1099, 0], [1050, 1099]], device="cuda")
    w = torch.rand((2, 2), device="cuda")
    y = layer.forward(x, ids, w, w1, w2, activation="relu")
    small = torch.tensor([[1, 0], [2, 1]], device="cuda")
    check_layer(y, x, small, w, w1[used].double(), w2[used].double(), False, "relu")


def test_refusals(layer, fp8):
    c = case(4, 2, 3, 64, 32, torch.bfloat16, True)
    args = [c["x"], c["ids"], c["weights"], c["w1"], c["w2"]]

    def call(i, value, **kw):
        return layer.forward(*[value if j == i else a for j, a in enumerate(args)], **{"gated": True, **kw})

    for i, value, error in ((0, c["x"].float(), TypeError), (1, c["ids"].float(), TypeError),
                            (1, c["ids"][:2], ValueError), (2, c["weights"].double(), TypeError),
                            (2, c["weights"][:, :1].contiguous(), ValueError), (3, c["w1"][:, :, :32], ValueError),
                            (4, c["w2"].transpose(1, 2), ValueError), (4, c["w2"][:2], ValueError),
                            (4, fp8.quantize(c["w2"], "blocks"), TypeError), (3, c["w1"][:, :63], ValueError)):
        with pytest.raises(error):
            call(i, value)
    with pytest.raises(ValueError, match="activation"):
        call(0, c["x"], activation="tanh")
    with pytest.raises(ValueError, match="pairs"):
        layer.forward(torch.zeros((300, 64), device="cuda"), torch.zeros((300, 2), dtype=torch.int64, device="cuda"),
                      torch.zeros((300, 2), device="cuda"), c["w1"].float(), c["w2"].float(), gated=True)

"""The 8-bit operators and the layer for a few tokens between other work on a stream: inputs written by the kernel right
before, calls captured in CUDA graphs, two streams at once; the calls of a training step together."""

import importlib.util
import os

import pytest
import torch

from tests.experts_harness import bound
from tests.fp8_harness import E5M2, meaning

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def mods():
    from dense_fp32_matrix_major_gb300 import experts, fp8, layer

    return experts, fp8, layer


def make(seed, tokens, width, hidden, E=3, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return {"x": torch.randn((tokens, width), generator=g, device="cuda").to(dtype),
            "dy": torch.randn((2 * tokens, hidden), generator=g, device="cuda").to(dtype),
            "ids": torch.randint(-1, E, (tokens, 2), generator=g, device="cuda"),
            "w": torch.rand((tokens, 2), generator=g, device="cuda"),
            "w1": (torch.randn((E, hidden, width), generator=g, device="cuda") * width ** -0.5).to(dtype),
            "w2": (torch.randn((E, width, hidden), generator=g, device="cuda") * hidden ** -0.5).to(dtype)}


def step(mods, s):
    """A layer's first product in 8 bits, forward and backward, and a decoding step."""
    experts, fp8, layer = mods
    E = s["w1"].shape[0]
    r = experts.sort(s["ids"], E)
    xs = experts.gather(s["x"], r)
    w8 = fp8.quantize(s["w1"], "blocks")
    y = fp8.gemm(fp8.quantize(xs, "rows"), w8, r.offsets, transB=True, dtype=s["x"].dtype)
    dx = fp8.gemm(fp8.quantize(s["dy"], "rows", dtype=E5M2), w8, r.offsets, dtype=s["x"].dtype)
    dw = fp8.gemm_wgrad(fp8.quantize(s["dy"], "columns", dtype=E5M2, offsets=r.offsets),
                        fp8.quantize(xs, "columns", offsets=r.offsets), r.offsets)
    dense = fp8.gemm(fp8.quantize(s["x"], "rows"), fp8.Quantized(w8.values[0], w8.scales[0]), transB=True)
    few = slice(0, min(8, s["x"].shape[0]))
    one = layer.forward(s["x"][few], s["ids"][few], s["w"][few], s["w1"], s["w2"])
    two = layer.forward(s["x"][few], s["ids"][few], s["w"][few], w8, fp8.quantize(s["w2"], "blocks"))
    return y, dx, dw, dense, one, two


def equal(got, want, what):
    for i, (a, b) in enumerate(zip(got, want)):
        assert torch.equal(a, b), (what, i)


@pytest.mark.parametrize("tokens", [5, 700])
def test_inputs_that_are_just_written(mods, tokens):
    sets = [make(i, tokens, 264, 136) for i in range(3)]
    want = []
    for s in sets:
        want.append(step(mods, s))
        torch.cuda.synchronize()
    now = {k: torch.zeros_like(v) for k, v in sets[0].items()}
    got = []
    for n in range(12):
        for k, v in sets[n % 3].items():
            now[k].copy_(v)
        got.append(step(mods, now))
    for n, g in enumerate(got):
        equal(g, want[n % 3], n)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_captured_in_graphs(mods, dtype):
    """Two graphs of the same calls on other data, replayed in turn and at once on two streams."""
    fixed = [make(i, 300, 264, 136, dtype=dtype) for i in range(2)]
    for s in fixed:
        step(mods, s)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for s in fixed:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(step(mods, s))
        graphs.append(graph)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for n in range(3):
        for i, s in enumerate(fixed):
            for k, v in make(10 + 2 * n + i, 300, 264, 136, dtype=dtype).items():
                s[k].copy_(v)
        torch.cuda.synchronize()
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for s, out in zip(fixed, outs):
            equal(out, step(mods, s), n)


def test_two_streams_at_once(mods):
    jobs = [make(1, 500, 520, 264), make(2, 400, 264, 136, dtype=torch.float32)]
    want = [step(mods, j) for j in jobs]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], [[], []]
    for _ in range(8):
        for s, j, out in zip(streams, jobs, got):
            with torch.cuda.stream(s):
                out.append(step(mods, j))
    torch.cuda.synchronize()
    for w, outs in zip(want, got):
        for o in outs:
            equal(o, w, "stream")


def test_gradients_in_slices_captured_and_on_two_streams(mods):
    """Few matrices over many rows, whose sums of slices lie in pool memory: in two graphs that are replayed at once, and
    eagerly on two streams."""
    fp8 = mods[1]
    off = [None, torch.tensor([0, 3000, 3000, 8100], dtype=torch.int32, device="cuda")]

    def operands(seed, offsets):
        g = torch.Generator(device="cuda").manual_seed(seed)
        return [fp8.quantize(torch.randn((8200, n), generator=g, device="cuda"), "columns", offsets=offsets)
                for n in (130, 270)]

    from dense_fp32_matrix_major_gb300 import sgemm

    fixed, graphs, outs = [operands(i, o) for i, o in enumerate(off)], [], []
    for (a, b), o in zip(fixed, off):
        fp8.gemm_wgrad(a, b, o)
        assert sgemm.last_launch_count() == 2  # slices, and their join
    torch.cuda.synchronize()
    for (a, b), o in zip(fixed, off):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(fp8.gemm_wgrad(a, b, o))
        graphs.append(graph)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for n in range(4):
        for i, (pair, o) in enumerate(zip(fixed, off)):
            for mine, new in zip(pair, operands(10 + 2 * n + i, o)):
                mine.values.view(torch.uint8).copy_(new.values.view(torch.uint8))
                mine.scales.copy_(new.scales)
        want = [fp8.gemm_wgrad(a, b, o) for (a, b), o in zip(fixed, off)]
        torch.cuda.synchronize()
        for out in outs:
            out.fill_(float("nan"))
        torch.cuda.synchronize()
        for _ in range(3):
            for graph, stream in zip(graphs, streams):
                with torch.cuda.stream(stream):
                    graph.replay()
        torch.cuda.synchronize()
        equal(outs, want, n)
        got = [[], []]
        for _ in range(6):
            for i, stream in enumerate(streams):
                with torch.cuda.stream(stream):
                    got[i].append(fp8.gemm_wgrad(*fixed[i], off[i]))
        torch.cuda.synchronize()
        for i in range(2):
            equal(got[i], [want[i]] * 6, (n, "eager"))


def test_stream_argument(mods):
    experts, fp8, layer = mods
    s = make(4, 64, 264, 136)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    a = fp8.quantize(s["x"], "rows", stream=stream)
    b = fp8.quantize(s["w1"][0], "blocks", stream=stream)
    y = fp8.gemm(a, b, transB=True, stream=stream)
    x, z = (fp8.quantize(t, "columns", stream=stream) for t in (s["x"], s["dy"][:64]))
    dw = fp8.gemm_wgrad(z, x, stream=stream)
    few = layer.forward(s["x"], s["ids"], s["w"], s["w1"], s["w2"], stream=stream)
    stream.synchronize()
    assert torch.equal(y, fp8.gemm(a, b, transB=True)) and torch.equal(dw, fp8.gemm_wgrad(z, x))
    assert torch.equal(few, layer.forward(s["x"], s["ids"], s["w"], s["w1"], s["w2"]))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_decoding_and_the_layer_of_many_tokens_agree(mods, dtype):
    """The layer for a few tokens against sort, gather, two products per expert and combine of the same weights."""
    experts, _, layer = mods
    s = make(9, 40, 264, 136, E=5, dtype=dtype)
    r = experts.sort(s["ids"], 5)
    pre = experts.gemm(experts.gather(s["x"], r), s["w1"], r.offsets, transB=True)
    h = experts.gemm(torch.nn.functional.silu(pre), s["w2"], r.offsets, transB=True)
    many = experts.combine(h, s["w"], r).double()
    few = layer.forward(s["x"], s["ids"], s["w"], s["w1"], s["w2"]).double()
    # Four roundings to 16 bits on the one way, one on the other: half a step each, on values of the result's size.
    step_of = torch.finfo(dtype).eps / 2
    assert float((few - many).norm() / many.norm()) <= 5 * step_of


def _example():
    spec = importlib.util.spec_from_file_location("fp8_layer", os.path.join(ROOT, "examples", "fp8_layer.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_example_runs():
    errors = _example().main(["--tokens", "300", "--experts", "4", "--width", "192", "--hidden", "320"])
    # Rounding to e4m3 is off by 2^-4 of a value at most, to e5m2 by 2^-3; a result's error over its norm is below
    # that of one factor plus the other, carried through two products and a gradient's.
    assert errors["y"] <= 3 * 2.0 ** -4 and errors["decode"] <= 4 * 2.0 ** -4
    assert all(errors[k] <= 2.0 ** -3 + 4 * 2.0 ** -4 for k in ("dx", "dw1", "dw2"))


def test_example_gradients():
    """The example's autograd functions against the formulas on the quantised operands, which they must meet to the
    bound of their sums."""
    from dense_fp32_matrix_major_gb300 import fp8

    ex = _example()
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((200, 192), generator=g, device="cuda").bfloat16().requires_grad_()
    w = (torch.randn((3, 160, 192), generator=g, device="cuda") * 0.1).requires_grad_()
    off = torch.tensor([0, 50, 50, 180], dtype=torch.int32, device="cuda")
    y = ex.ExpertLinear.apply(x, w, off)
    dy = torch.randn((200, 160), generator=g, device="cuda").bfloat16()
    dx, dw = torch.autograd.grad(y, (x, w), dy)
    wq = meaning(fp8.quantize(w.detach(), "blocks"), "blocks")
    dyq = meaning(fp8.quantize(dy, "rows", dtype=E5M2), "rows")
    for e, (a, b) in enumerate(((0, 50), (50, 50), (50, 180))):
        exact, size = (dyq[a:b] @ wq[e]).cpu().numpy(), (dyq[a:b].abs() @ wq[e].abs()).cpu().numpy()
        off_by = abs(dx[a:b].double().cpu().numpy() - exact)
        assert (off_by <= bound(exact, size, 160, torch.bfloat16)).all()
    assert not dx[180:].any() and not dw[1].any() and dw.dtype == torch.float32
    graph = torch.cuda.CUDAGraph()  # forward and backward in one capture, leaves of their own
    leaves = [x.detach().clone().requires_grad_(), w.detach().clone().requires_grad_()]
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = torch.autograd.grad(ex.ExpertLinear.apply(*leaves, off), leaves, dy)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], dx) and torch.equal(got[1], dw)

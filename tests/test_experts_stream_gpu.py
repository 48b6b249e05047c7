"""The mixture-of-experts operators between other work on a stream: inputs written by the kernel right before, and
calls captured in a CUDA graph."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ex():
    from dense_fp32_matrix_major_gb300 import experts

    return experts


@pytest.mark.parametrize("tokens,top_k,experts", [(600, 2, 8), (5000, 2, 16), (16384, 8, 64)])
def test_sort_of_ids_that_are_just_written(ex, tokens, top_k, experts):
    g = torch.Generator(device="cuda").manual_seed(tokens)
    source = torch.randint(-1, experts, (40, tokens, top_k), generator=g, device="cuda")
    ids = torch.empty((tokens, top_k), dtype=torch.int64, device="cuda")
    got = []
    for one in source:
        ids.copy_(one)
        got.append(ex.sort(ids, experts))
    for one, r in zip(source, got):
        key = torch.where(one < 0, experts, one).reshape(-1)
        assert torch.equal(r.order.long(), torch.argsort(key, stable=True))
        assert r.offsets[-1] == (one >= 0).sum()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("K", [512, 8192])
def test_w4_matvec_of_inputs_that_are_just_written(ex, dtype, K):
    """Every input is written by the kernels before the call, x staying in shared memory or streamed."""
    g = torch.Generator(device="cuda").manual_seed(K)
    rows, N, E, group, sets = 12, 3000, 4, 128, 3
    xs = torch.randn((sets, rows, K), generator=g, device="cuda").to(dtype)
    qs = torch.randint(0, 256, (sets, E, N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = torch.rand((sets, E, N, K // group), generator=g, device="cuda")
    ids = torch.randint(-1, E, (sets, rows), generator=g, device="cuda", dtype=torch.int32)
    want = []
    for i in range(sets):
        want.append(ex.w4_matvec(xs[i], qs[i], scales[i], group=group, ids=ids[i]))
        torch.cuda.synchronize()
    x, q, s, at = (torch.zeros_like(t[0]) for t in (xs, qs, scales, ids))
    got = []
    for n in range(30):
        i = n % sets
        for to, source in ((x, xs), (q, qs), (s, scales), (at, ids)):
            to.copy_(source[i])
        got.append(ex.w4_matvec(x, q, s, group=group, ids=at))
    for n, y in enumerate(got):
        assert torch.equal(y, want[n % sets]), n


def step(ex, ids, x, w, b, q, scales):
    """A layer's calls, forward and backward, and a decoding step; with copies of unaligned operands, slices of a long
    sum and streamed x, which take memory from the library's pool."""
    r = ex.sort(ids, b.shape[0])
    xs = ex.gather(x, r)
    h = ex.gemm(xs, b, r.offsets)
    y = ex.combine(h, w, r)
    dh, dw = ex.combine_grad(y, h, w, r)
    dxs = ex.gemm(dh, b, r.offsets, transB=True)
    db = ex.gemm_wgrad(xs, dh, r.offsets)
    dx = ex.gather_grad(dxs, r)
    few = ex.w4_matvec(x[:5], q, scales, group=128)
    odd = ex.gemm(xs[:, 1:], b[:, 1:], r.offsets)
    sliced = ex.gemm_wgrad(xs[:, :64], dh, r.offsets)
    return r.order, xs, h, y, dh, dw, db, dx, few, odd, sliced


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("tokens", [6, 6000])
def test_captured_in_a_graph(ex, dtype, tokens):
    from dense_fp32_matrix_major_gb300 import sgemm

    g = torch.Generator(device="cuda").manual_seed(tokens)
    width, N, E = 6400, 96, 2

    def inputs():
        return (torch.randint(-1, E, (tokens, 2), generator=g, device="cuda"),
                torch.randn((tokens, width), generator=g, device="cuda").to(dtype),
                torch.rand((tokens, 2), generator=g, device="cuda"))

    b = (torch.randn((E, width, N), generator=g, device="cuda") * 0.01).to(dtype)
    q = torch.randint(0, 256, (300, width // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = torch.rand((300, width // 128), generator=g, device="cuda") * 0.01
    fixed = inputs()
    step(ex, *fixed, b, q, scales)  # the first calls set kernels up
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(ex, *fixed, b, q, scales)
    for _ in range(4):
        new = inputs()
        for to, source in zip(fixed, new):
            to.copy_(source)
        graph.replay()
        replayed = [t.clone() for t in out]
        want = step(ex, *new, b, q, scales)
        torch.cuda.synchronize()
        for i, (x, y) in enumerate(zip(replayed, want)):
            assert torch.equal(x, y), i
    assert sgemm.device_status() == 0


def test_two_streams_at_once(ex):
    """Calls on two streams that nothing orders: each has its own scratch and gives its own results."""
    g = torch.Generator(device="cuda").manual_seed(8)
    width, N, E = 6400, 96, 2
    jobs = []
    for tokens, dtype in ((700, torch.float32), (500, torch.bfloat16)):
        jobs.append((torch.randint(-1, E, (tokens, 2), generator=g, device="cuda"),
                     torch.randn((tokens, width), generator=g, device="cuda").to(dtype),
                     torch.rand((tokens, 2), generator=g, device="cuda"),
                     (torch.randn((E, width, N), generator=g, device="cuda") * 0.01).to(dtype),
                     torch.randint(0, 256, (300, width // 2), generator=g, device="cuda", dtype=torch.uint8),
                     torch.rand((300, width // 128), generator=g, device="cuda") * 0.01))
    want = [step(ex, *j) for j in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(10):
        for s, j, out in zip(streams, jobs, got):
            with torch.cuda.stream(s):
                out.append(step(ex, *j))
    torch.cuda.synchronize()
    for w, outs in zip(want, got):
        for o in outs:
            for i, (x, y) in enumerate(zip(o, w)):
                assert torch.equal(x, y), i

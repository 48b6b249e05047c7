"""The mixture-of-experts operators between other work on a stream: inputs written by the kernel right before."""

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

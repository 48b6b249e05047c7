"""The binding's checks of where tensors are, without a GPU: tensors stand in that only know their device."""

import pytest
import torch


class On:
    def __init__(self, device, requires_grad=False):
        self.device_index, self.cuda_stream, self.requires_grad = device, 77, requires_grad

    def get_device(self):
        return self.device_index


@pytest.fixture
def ex(monkeypatch):
    from dense_fp32_matrix_major_gb300 import _build

    _build.build()
    from dense_fp32_matrix_major_gb300 import experts

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    return experts


def test_every_tensor_is_on_the_current_device(ex):
    assert ex._stream_handle(On(0), On(0), None, On(0)) == 77
    for tensors in ((On(1),), (On(0), On(1)), (On(0), None, On(0), On(2))):
        with pytest.raises(ValueError, match="current device"):
            ex._stream_handle(On(0), *tensors)
    with pytest.raises(ValueError, match="stream"):
        ex._stream_handle(On(1), On(0))


def test_calls_check_every_tensor(ex, monkeypatch):
    """Each call hands all its tensors to the check, outputs and routing among them."""
    seen = []

    class Stop(Exception):
        pass

    def check(stream, *tensors):
        seen.append(tensors)
        raise Stop

    monkeypatch.setattr(ex, "_stream_handle", check)
    monkeypatch.setattr(ex, "_rows", lambda t, name, dtype=None: (0, t.shape[1]))
    monkeypatch.setattr(ex, "_matrices", lambda t, name, dtype: (t.shape[2], t.shape[1] * t.shape[2]))
    monkeypatch.setattr(ex, "_contiguous", lambda t, *rest: 0)
    i32 = {"dtype": torch.int32}
    r = ex.Routing(torch.zeros(3, **i32), torch.zeros(8, **i32), torch.zeros(4, 2, **i32))
    x, h, w, y = torch.zeros(4, 8), torch.zeros(8, 8), torch.zeros(4, 2), torch.zeros(4, 8)
    b, q, s, z = torch.zeros(2, 8, 6), torch.zeros(2, 5, 4), torch.zeros(2, 5, 1), torch.zeros(2, 5, 1)
    ids, c, y5 = torch.zeros(4), torch.zeros(8, 6), torch.zeros(4, 5)
    for call, tensors in (
        (lambda: ex.gather(x, r, out=h), (x, h, r.slot, r.offsets)),
        (lambda: ex.combine(h, w, r, out=y), (h, w, y, r.slot, r.offsets)),
        (lambda: ex.gather_grad(h, r, out=y), (h, y, r.slot, r.offsets)),
        (lambda: ex.combine_grad(y, h, w, r), (y, h, w, r.slot, r.offsets)),
        (lambda: ex.gemm(h, b, r.offsets, out=c), (h, b, r.offsets, c)),
        (lambda: ex.gemm_wgrad(h, c, r.offsets, out=b), (h, c, r.offsets, b)),
        (lambda: ex.w4_matvec(x, q, s, group=32, zeros=z, ids=ids, out=y5), (x, q, s, z, ids, y5)),
    ):
        with pytest.raises(Stop):
            call()
        got = seen.pop()
        assert all(any(t is g for g in got) for t in tensors)


def test_a_lost_gradient_draws_a_warning(ex):
    import warnings

    with pytest.warns(UserWarning, match="cut from the graph"):
        ex._stream_handle(On(0), On(0), None, On(0, requires_grad=True))
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        ex._stream_handle(On(0), On(0), None, On(0))
        with torch.no_grad():
            ex._stream_handle(On(0), On(0, requires_grad=True))

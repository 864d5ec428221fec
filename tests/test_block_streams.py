"""stream= of the operators around the projections, without a GPU: a stream of another device than the tensors' is
refused (the call would run on that device's current stream instead)."""
import pytest

torch = pytest.importorskip("torch")


class Stream:
    """As much of a stream as is looked at before it is made current."""

    def __init__(self, device):
        self.device = torch.device(device)


class OnDevice(torch.Tensor):
    """A tensor that says it is on a GPU."""

    device = torch.device("cuda", 0)


@pytest.fixture
def calls():
    from bit_rank_compensated_b200 import svdq

    def on(*shape, dtype=torch.float32):
        return torch.zeros(*shape, dtype=dtype).as_subclass(OnDevice)

    x, q, one, pos = on(4, 32), on(4, 2, 16), on(4), on(4, 2)
    i8, axes = on(4, 32, dtype=torch.int8), svdq.RopeAxes((4, 4))
    return svdq, [
        lambda s: svdq.layer_norm(x, stream=s), lambda s: svdq.layer_norm_backward(x, x, one, one, stream=s),
        lambda s: svdq.i8_quantize_rows(x, stream=s), lambda s: svdq.i8_layer_norm_quantize(x, stream=s),
        lambda s: svdq.i8_gemm(i8, one, i8, one, stream=s), lambda s: svdq.i8_linear_forward(x, i8, one, stream=s),
        lambda s: svdq.rope_axes_table(pos, axes, stream=s), lambda s: svdq.rope_axes_apply(q, None, pos, axes, stream=s),
    ]


def test_a_stream_of_another_device_is_refused(calls, monkeypatch):
    svdq, fs = calls
    made_current = []
    monkeypatch.setattr(torch.cuda, "stream", lambda s: made_current.append(s) or (_ for _ in ()).throw(KeyError))
    for f in fs:
        with pytest.raises(ValueError, match="cuda:1.*cuda:0"):
            f(Stream("cuda:1"))
        assert not made_current
    # and one of the tensors' device is made current
    for f in fs:
        with pytest.raises(KeyError):
            f(Stream("cuda:0"))
    assert len(made_current) == len(fs)

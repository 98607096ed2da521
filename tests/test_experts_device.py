"""The expert operators on a device that is not the current one, on the host:
tensors that say they are on cuda:1 while cuda:0 is current, and a library that
notes which device is current when it is called.  No kernel runs here."""
import contextlib

import pytest

torch = pytest.importorskip("torch")

HERE = torch.device("cuda", 1)


class OnGpu1(torch.Tensor):
    device = property(lambda self: HERE)
    is_cuda = property(lambda self: True)


def tensor(*shape, dtype=torch.float16):
    return torch.zeros(*shape, dtype=dtype).as_subclass(OnGpu1)


@pytest.fixture
def seen(monkeypatch):
    import distance_argmin_gb300 as km
    state = {"current": 0, "calls": []}

    @contextlib.contextmanager
    def device(d):
        before, state["current"] = state["current"], d if isinstance(d, int) else d.index
        yield
        state["current"] = before

    class Library:
        def __getattr__(self, name):
            def call(*args):
                state["calls"].append((name, state["current"], args[-1]))
                return km.KMEANS_OK
            return call

    monkeypatch.setattr(km, "_lib", Library())
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: state["current"], raising=False)
    monkeypatch.setattr(torch.cuda, "device", device)
    # a handle per device, as the default streams do not have
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 1000 + index, raising=False)
    return km, state


def calls(km):
    i32, f32, u8 = torch.int32, torch.float32, torch.uint8
    x, xs, wts = tensor(4, 8), tensor(8, 8), tensor(4, 2, dtype=f32)
    rows, offsets, ws = tensor(4, 2, dtype=i32), tensor(4, dtype=i32), tensor(256, dtype=u8)
    w = tensor(3, 8, 8)
    return {
        "kmeans_route": lambda: km.kmeans_route(rows, 3, offsets, tensor(8, dtype=i32), rows, ws),
        "kmeans_route_gather": lambda: km.kmeans_route_gather(x, rows, offsets, xs),
        "kmeans_route_combine": lambda: km.kmeans_route_combine(xs, rows, offsets, wts, None, x),
        "kmeans_route_combine_grad": lambda: km.kmeans_route_combine_grad(x, xs, rows, offsets, wts, xs, wts),
        "kmeans_linear": lambda: km.kmeans_linear(x, w, offsets=offsets, y=x, ws=ws),
        "kmeans_linear_grad": lambda: km.kmeans_linear_grad(x, x, w, offsets=offsets, need_dw=False, need_db=False,
                                                            dx=x, ws=ws),
    }


@pytest.mark.parametrize("name", ["kmeans_route", "kmeans_route_gather", "kmeans_route_combine",
                                  "kmeans_route_combine_grad", "kmeans_linear", "kmeans_linear_grad"])
@pytest.mark.parametrize("current", [0, 1])
def test_the_tensors_device_is_current_during_the_call(seen, name, current):
    km, state = seen
    state["current"] = current
    calls(km)[name]()
    assert state["calls"] == [(name, 1, 1001)]
    assert state["current"] == current


def test_a_stream_of_another_device_is_refused(seen, monkeypatch):
    km, state = seen

    class Stream:
        device = torch.device("cuda", 0)

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    x, rows, offsets = tensor(4, 8), tensor(4, 2, dtype=torch.int32), tensor(4, dtype=torch.int32)
    from distance_argmin_gb300 import experts
    for call in (lambda: km.kmeans_route_gather(x, rows, offsets, stream=Stream()),
                 lambda: experts.experts_forward(x, rows, x, x, stream=Stream())):
        with pytest.raises(ValueError, match="stream is on cuda:0"):
            call()
    assert not state["calls"]
    with pytest.raises(ValueError, match="CUDA device"):
        experts.experts_forward(torch.zeros(4, 8), rows, x, x)


def test_a_stream_handle_is_taken_as_one_of_the_tensors_device(seen, monkeypatch):
    km, state = seen
    made = []
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device: made.append((handle, device)) or "stream")
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    x, xs = tensor(4, 8), tensor(8, 8)
    km.kmeans_route_gather(x, tensor(4, 2, dtype=torch.int32), tensor(4, dtype=torch.int32), xs, stream=77)
    assert made == [(77, HERE)]

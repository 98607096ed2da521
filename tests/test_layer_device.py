"""The gate, the layer norm and the cross entropy on a device that is not the
current one, on the host: tensors that say they are on cuda:1 while cuda:0 is
current, and a library that notes which device is current when it is called.
The binding's refusals of wrong arguments are seen here too.  No kernel runs."""
import contextlib

import pytest

torch = pytest.importorskip("torch")

HERE = torch.device("cuda", 1)
I32, I64, F32, F16, U8 = torch.int32, torch.int64, torch.float32, torch.float16, torch.uint8


class OnGpu1(torch.Tensor):
    device = property(lambda self: HERE)
    is_cuda = property(lambda self: True)


def tensor(*shape, dtype=F16):
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
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 1000 + index, raising=False)
    return km, state


def calls(km, **other):
    """The calls, with some arguments replaced."""
    def a(name, value):
        return other.get(name, value)

    x, v, ws = a("x", tensor(4, 8)), a("v", tensor(4, dtype=F32)), a("ws", tensor(256, dtype=U8))
    ids, wts = a("ids", tensor(4, 2, dtype=I32)), a("wts", tensor(4, 2, dtype=F32))
    w, labels, vec = a("w", tensor(5, 8)), a("labels", tensor(4, dtype=I64)), a("vec", tensor(8))
    return {
        "kmeans_gate": lambda: km.kmeans_gate(x, a("topk", 2), scores=a("scores", "softmax"), bias=a("bias", None),
                                              groups=a("groups", 1), topk_groups=a("topk_groups", None),
                                              scale=a("scale", 1.0), ids=ids, weights=wts),
        "kmeans_gate_grad": lambda: km.kmeans_gate_grad(wts, x, ids, scores=a("scores", "softmax"),
                                                        scale=a("scale", 1.0), dlogits=a("out", x)),
        "kmeans_layernorm": lambda: km.kmeans_layernorm(x, vec, vec, eps=a("eps", 1e-5), y=a("out", x), mean=v, rstd=v),
        "kmeans_layernorm_grad": lambda: km.kmeans_layernorm_grad(a("dy", x), x, v, v, weight=vec,
                                                                  residual=a("residual", None), dx=a("out", x),
                                                                  dweight=vec, dbias=vec, ws=ws),
        "kmeans_cross_entropy": lambda: km.kmeans_cross_entropy(x, w, labels, scale=a("scale", 1.0), loss=v, lse=v,
                                                                ws=ws),
        "kmeans_cross_entropy_grad": lambda: km.kmeans_cross_entropy_grad(v, x, w, labels, v, scale=a("scale", 1.0),
                                                                          dx=a("out", x), dw=w, ws=ws),
    }


NAMES = list(calls(None))


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("current", [0, 1])
def test_the_tensors_device_is_current_during_the_call(seen, name, current):
    km, state = seen
    state["current"] = current
    calls(km)[name]()
    assert state["calls"] == [(name, 1, 1001)]
    assert state["current"] == current


@pytest.mark.parametrize("name", NAMES)
def test_a_stream_of_another_device_is_refused(seen, monkeypatch, name):
    km, state = seen

    class Stream:
        device = torch.device("cuda", 0)

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    x, v, i = tensor(4, 8), tensor(4, dtype=F32), tensor(4, 2, dtype=I32)
    call = {"kmeans_gate": lambda s: km.kmeans_gate(x, 2, stream=s),
            "kmeans_gate_grad": lambda s: km.kmeans_gate_grad(i.float().as_subclass(OnGpu1), x, i, stream=s),
            "kmeans_layernorm": lambda s: km.kmeans_layernorm(x, stream=s),
            "kmeans_layernorm_grad": lambda s: km.kmeans_layernorm_grad(x, x, v, v, stream=s),
            "kmeans_cross_entropy": lambda s: km.kmeans_cross_entropy(x, x, v, stream=s),
            "kmeans_cross_entropy_grad": lambda s: km.kmeans_cross_entropy_grad(v, x, x, v, v, stream=s)}[name]
    with pytest.raises(ValueError, match="stream is on cuda:0"):
        call(Stream())
    assert not state["calls"]


@pytest.mark.parametrize("name,wrong,error", [
    ("kmeans_gate", dict(topk=9), "topk"), ("kmeans_gate", dict(topk=-1), "topk"),
    ("kmeans_gate", dict(scores="max"), "scores"), ("kmeans_gate", dict(groups=3), "groups"),
    ("kmeans_gate", dict(groups=2, topk_groups=3), "topk_groups"), ("kmeans_gate", dict(scale=float("nan")), "scale"),
    ("kmeans_gate", dict(bias=tensor(7, dtype=F32)), "bias"), ("kmeans_gate", dict(x=tensor(4, 8, 1)), "logits"),
    ("kmeans_gate", dict(ids=tensor(4, 3, dtype=I32)), "ids"),
    ("kmeans_gate_grad", dict(ids=tensor(3, 2, dtype=I32)), "ids"),
    ("kmeans_gate_grad", dict(scale=float("inf")), "scale"), ("kmeans_gate_grad", dict(out=tensor(4, 7)), "dlogits"),
    ("kmeans_layernorm", dict(eps=-1.0), "eps"), ("kmeans_layernorm", dict(vec=tensor(7)), "weight"),
    ("kmeans_layernorm", dict(out=tensor(3, 8)), "y"), ("kmeans_layernorm", dict(v=tensor(3, dtype=F32)), "mean"),
    ("kmeans_layernorm_grad", dict(dy=tensor(4, 7)), "dy"), ("kmeans_layernorm_grad", dict(out=tensor(4, 7)), "dx"),
    ("kmeans_layernorm_grad", dict(residual=tensor(4, 9)), "residual"),
    ("kmeans_cross_entropy", dict(w=tensor(5, 7)), "features"), ("kmeans_cross_entropy", dict(scale=0.0), "scale"),
    ("kmeans_cross_entropy", dict(labels=tensor(3, dtype=I64)), "labels"),
    ("kmeans_cross_entropy", dict(w=tensor(8)), "w must be"),
    ("kmeans_cross_entropy_grad", dict(out=tensor(4, 7)), "dx"),
    ("kmeans_cross_entropy_grad", dict(v=tensor(5, dtype=F32)), "dloss"),
])
def test_wrong_shapes_and_values_are_refused(seen, name, wrong, error):
    km, state = seen
    state["current"] = 1
    with pytest.raises(ValueError, match=error):
        calls(km, **wrong)[name]()
    assert not state["calls"]


@pytest.mark.parametrize("name,wrong", [
    ("kmeans_gate", dict(x=tensor(4, 8, dtype=torch.float64))), ("kmeans_gate", dict(bias=tensor(8))),
    ("kmeans_gate_grad", dict(wts=tensor(4, 2))), ("kmeans_gate_grad", dict(ids=tensor(4, 2, dtype=I64))),
    ("kmeans_layernorm", dict(vec=tensor(8, dtype=F32))), ("kmeans_layernorm", dict(v=tensor(4))),
    ("kmeans_layernorm_grad", dict(dy=tensor(4, 8, dtype=F32))), ("kmeans_layernorm_grad", dict(ws=tensor(256))),
    ("kmeans_cross_entropy", dict(w=tensor(5, 8, dtype=torch.bfloat16))),
    ("kmeans_cross_entropy", dict(labels=tensor(4, dtype=F32))), ("kmeans_cross_entropy_grad", dict(v=tensor(4))),
])
def test_wrong_types_are_refused(seen, name, wrong):
    km, state = seen
    state["current"] = 1
    with pytest.raises(TypeError):
        calls(km, **wrong)[name]()
    assert not state["calls"]

"""Out-of-bounds writes, uninitialised reads, stream order, captured graphs and
other streams of the gate, the layer norm and the cross entropy.

Every workspace and output sits between two canary-filled guard regions; outputs
start poisoned and the workspace as 0xFF bytes.  After each call the guards must
be intact and the results equal, bit for bit, those of a call on fresh buffers.
Inputs lie between NaN values in memory.
"""
import pytest

from test_experts_guards import Guarded, fenced, like, normal, same

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

DTYPES = [torch.float32, torch.float16, torch.bfloat16]


def held(call, outs):
    """`call(*guarded outputs)` writes all of them, and no byte beside them."""
    ref = call(*[torch.empty_like(t) for t in outs])
    out = [like(t) for t in outs]
    call(*[o.t for o in out])
    assert all(o.intact() and same(o.t, r) for o, r in zip(out, ref))
    assert not any(bool(torch.isnan(o.t).any()) for o in out if o.t.dtype.is_floating_point)


def workspace(t):
    return Guarded((t.numel(),), torch.uint8, 0xFF)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,E,topk,groups", [(1, 3, 2, 1), (37, 65, 5, 5), (300, 256, 8, 8), (11, 1025, 9, 1), (5, 4096, 32, 32)])
def test_the_gate_stays_inside_its_buffers(gpu_lib, n, E, topk, groups, dtype):
    z, bias = fenced(normal((n, E), dtype, E)), fenced(normal((E,), torch.float32, 1, 0.1))
    dw = fenced(normal((n, topk), torch.float32, 2))
    ids, w = gpu_lib.kmeans_gate(z, topk, bias=bias, groups=groups, topk_groups=max(1, groups // 2))
    held(lambda i, v: gpu_lib.kmeans_gate(z, topk, bias=bias, groups=groups, topk_groups=max(1, groups // 2), ids=i,
                                          weights=v), [ids, w])
    for renormalize in (False, True):
        held(lambda d: [gpu_lib.kmeans_gate_grad(dw, z, ids, renormalize=renormalize, dlogits=d)], [torch.empty_like(z)])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,d", [(1, 1), (3, 7), (50, 64), (70, 33), (300, 255), (41, 1031), (90, 2048), (20, 8200), (3, 40001)])
def test_the_layer_norm_stays_inside_its_buffers(gpu_lib, n, d, dtype):
    x, dy, res = (fenced(normal((n, d), dtype, s)) for s in (1, 2, 3))
    w, b = fenced(normal((d,), dtype, 4)), fenced(normal((d,), dtype, 5))
    y, mean, rstd = gpu_lib.kmeans_layernorm(x, w, b, save_stats=True)
    held(lambda *o: gpu_lib.kmeans_layernorm(x, w, b, y=o[0], mean=o[1], rstd=o[2]), [y, mean, rstd])
    size = gpu_lib.layernorm_workspace(n, d)
    for residual in (None, res):
        ws = workspace(size)
        held(lambda *o: gpu_lib.kmeans_layernorm_grad(dy, x, mean, rstd, weight=w, residual=residual, dx=o[0],
                                                      dweight=o[1], dbias=o[2], ws=ws.t), [x, w, b])
        assert ws.intact() and gpu_lib.kmeans_device_status(ws.t) == gpu_lib.KMEANS_OK


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (3, 40, 9), (64, 1000, 72), (65, 257, 40), (300, 4097, 515), (700, 129, 264),
                                   (5000, 300, 64), (40, 70001, 24)])
def test_the_cross_entropy_stays_inside_its_buffers(gpu_lib, m, n, k, dtype):
    x, w = fenced(normal((m, k), dtype, 1)), fenced(normal((n, k), dtype, 2, k ** -0.5))
    g = torch.Generator(device="cuda")
    g.manual_seed(m)
    labels = torch.randint(-1, n, (m,), generator=g, device="cuda")
    dloss = fenced(torch.rand(m, generator=g, device="cuda"))
    v = torch.empty(m, device="cuda")
    ws = workspace(gpu_lib.cross_entropy_workspace(gpu_lib.OP_CROSS_ENTROPY, m, n, k))
    held(lambda a, b: gpu_lib.kmeans_cross_entropy(x, w, labels, loss=a, lse=b, ws=ws.t), [v, v])
    assert ws.intact() and gpu_lib.kmeans_device_status(ws.t) == gpu_lib.KMEANS_OK
    _, lse = gpu_lib.kmeans_cross_entropy(x, w, labels)
    lse = fenced(lse)
    ws = workspace(gpu_lib.cross_entropy_workspace(gpu_lib.OP_CROSS_ENTROPY_GRAD, m, n, k))
    held(lambda a, b: gpu_lib.kmeans_cross_entropy_grad(dloss, x, w, labels, lse, dx=a, dw=b, ws=ws.t), [x, w])
    assert ws.intact() and gpu_lib.kmeans_device_status(ws.t) == gpu_lib.KMEANS_OK


def chain(km, x, wg, w, labels, bias, ws=None):
    """Every operator once, one on the other's results."""
    m, d = x.shape
    y, mean, rstd = km.kmeans_layernorm(x, save_stats=True)
    logits, _ = km.kmeans_linear(y, wg)
    ids, weights = km.kmeans_gate(logits, 3, bias=bias, groups=4, topk_groups=2)
    dlogits = km.kmeans_gate_grad(weights, logits, ids)
    loss, lse = km.kmeans_cross_entropy(y, w, labels, ws=ws)
    dx, dw = km.kmeans_cross_entropy_grad(loss, y, w, labels, lse, ws=ws)
    dn, dg, db = km.kmeans_layernorm_grad(dx, x, mean, rstd, residual=y)
    return y, mean, rstd, ids, weights, dlogits, loss, lse, dx, dw, dn, dg, db


def chain_inputs(seed, m=700, d=256, n=5000, E=32):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x, wg, w = normal((m, d), torch.bfloat16, seed), normal((E, d), torch.bfloat16, 7, d ** -0.5), \
        normal((n, d), torch.bfloat16, 8, d ** -0.5)
    return x, wg, w, torch.randint(-1, n, (m,), generator=g, device="cuda"), normal((E,), torch.float32, 9, 0.05)


def test_each_call_sees_what_was_written_just_before_it(gpu_lib):
    big = normal((4096, 4096), torch.float32, 9)
    for seed in range(3):
        x, *rest = chain_inputs(seed)
        torch.cuda.synchronize()
        want = chain(gpu_lib, x, *rest)
        torch.cuda.synchronize()
        late = torch.zeros_like(x)
        (big @ big).mean()  # keeps the stream busy
        late.copy_(x)
        got = chain(gpu_lib, late, *rest)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_captured_calls_replay_on_new_inputs(gpu_lib):
    """A captured chain, replayed on other values in the same buffers, with an eager chain of its own workspace
    between the replays."""
    args = chain_inputs(1)
    x, labels = args[0], args[3]
    ws = gpu_lib.cross_entropy_workspace(gpu_lib.OP_CROSS_ENTROPY_GRAD, x.shape[0], args[2].shape[0], x.shape[1])
    chain(gpu_lib, *args, ws=ws)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        out = chain(gpu_lib, *args, ws=ws)
    for seed in (2, 3):
        other = chain_inputs(seed)
        want = chain(gpu_lib, *other)
        x.copy_(other[0])
        labels.copy_(other[3])
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
        assert gpu_lib.kmeans_device_status(ws) == gpu_lib.KMEANS_OK


def test_calls_on_two_streams_at_once(gpu_lib):
    inputs = [chain_inputs(s) for s in (4, 5)]
    want = [chain(gpu_lib, *a) for a in inputs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in inputs]
    for _ in range(5):
        got = []
        for a, s in zip(inputs, streams):
            with torch.cuda.stream(s):
                got.append(chain(gpu_lib, *a))
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(g, w))


def test_the_stream_argument(gpu_lib):
    x, wg, w, labels, bias = chain_inputs(6)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    logits = normal((700, 32), torch.bfloat16, 3)
    pairs = [(gpu_lib.kmeans_layernorm(x, save_stats=True), gpu_lib.kmeans_layernorm(x, save_stats=True, stream=s)),
             (gpu_lib.kmeans_gate(logits, 3, bias=bias), gpu_lib.kmeans_gate(logits, 3, bias=bias, stream=s)),
             (gpu_lib.kmeans_cross_entropy(x, w, labels), gpu_lib.kmeans_cross_entropy(x, w, labels, stream=s.cuda_stream))]
    _, mean, rstd = pairs[0][0]
    ids, weights = pairs[1][0]
    loss, lse = pairs[2][0]
    s.wait_stream(torch.cuda.current_stream())
    pairs += [(gpu_lib.kmeans_layernorm_grad(x, x, mean, rstd), gpu_lib.kmeans_layernorm_grad(x, x, mean, rstd, stream=s)),
              ([gpu_lib.kmeans_gate_grad(weights, logits, ids)], [gpu_lib.kmeans_gate_grad(weights, logits, ids, stream=s)]),
              (gpu_lib.kmeans_cross_entropy_grad(loss, x, w, labels, lse),
               gpu_lib.kmeans_cross_entropy_grad(loss, x, w, labels, lse, stream=s))]
    torch.cuda.synchronize()
    for a, b in pairs:
        assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_offsets_past_32_bits(gpu_lib):
    """Tensors of more than 2^31 values: the last rows are what they are alone."""
    n, d = 2 ** 20 + 3, 2056
    x = torch.empty((n, d), dtype=torch.bfloat16, device="cuda")
    tail = normal((5, d), torch.bfloat16, 1)
    x.zero_()
    x[-5:] = tail
    y, mean, rstd = gpu_lib.kmeans_layernorm(x, save_stats=True)
    want = gpu_lib.kmeans_layernorm(tail, save_stats=True)
    assert torch.equal(y[-5:], want[0]) and torch.equal(mean[-5:], want[1]) and torch.equal(rstd[-5:], want[2])
    dx, dw, db = gpu_lib.kmeans_layernorm_grad(x, x, mean, rstd, dx=y)
    alone = gpu_lib.kmeans_layernorm_grad(tail, tail, want[1], want[2])
    assert torch.equal(dx[-5:], alone[0])
    del y, dx
    ids, w = gpu_lib.kmeans_gate(x, 4)
    got = gpu_lib.kmeans_gate(tail, 4)
    assert torch.equal(ids[-5:], got[0]) and torch.equal(w[-5:], got[1])
    dl = gpu_lib.kmeans_gate_grad(w, x, ids, renormalize=False)
    assert torch.equal(dl[-5:], gpu_lib.kmeans_gate_grad(got[1], tail, got[0], renormalize=False))
    del dl
    labels = torch.full((n,), -1, device="cuda")
    labels[-5:] = torch.tensor([1, 0, 2, 1, 0], device="cuda")
    classes = normal((3, d), torch.bfloat16, 2, d ** -0.5)
    loss, lse = gpu_lib.kmeans_cross_entropy(x, classes, labels)
    one = gpu_lib.kmeans_cross_entropy(tail, classes, labels[-5:].contiguous())
    assert not loss[:-5].any() and torch.allclose(loss[-5:], one[0], rtol=1e-5, atol=1e-5)
    dx, dw = gpu_lib.kmeans_cross_entropy_grad(torch.ones(n, device="cuda"), x, classes, labels, lse)
    few = gpu_lib.kmeans_cross_entropy_grad(torch.ones(5, device="cuda"), tail, classes, labels[-5:].contiguous(), one[1])
    assert not dx[:-5].any() and torch.allclose(dx[-5:].float(), few[0].float(), rtol=0.02, atol=1e-3)
    assert torch.allclose(dw.float(), few[1].float(), rtol=0.02, atol=1e-2)

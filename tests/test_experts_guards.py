"""Out-of-bounds writes, uninitialised reads and stream order of the expert
routing and the products.

Every workspace and output here sits between two canary-filled guard regions;
outputs start poisoned and the workspace as 0xFF bytes.  After each call the
guards must be intact and the results equal, bit for bit, those of a call on
fresh buffers, so a write past a buffer, a skipped output or a read of scratch
that the call did not initialise shows up.  Inputs lie at the end of their own
guarded buffers, between NaN rows.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

GUARD = 64 * 1024  # bytes on each side
CANARY = 0xA5


class Guarded:
    def __init__(self, shape, dtype, fill):
        nbytes = int(np.prod(shape)) * torch.empty((), dtype=dtype).element_size()
        room = (nbytes + 255) // 256 * 256
        self.raw = torch.full((2 * GUARD + room,), CANARY, dtype=torch.uint8, device="cuda")
        self.nbytes = nbytes
        self.t = self.raw[GUARD:GUARD + nbytes].view(dtype).view(shape)
        self.t.fill_(fill)

    def intact(self):
        torch.cuda.synchronize()
        return bool((self.raw[:GUARD] == CANARY).all()) and bool((self.raw[GUARD + self.nbytes:] == CANARY).all())


def like(t):
    return Guarded(tuple(t.shape), t.dtype, float("nan") if t.dtype.is_floating_point else -7)


def same(a, b):
    return a.cpu().contiguous().view(torch.uint8).numpy().tobytes() == b.cpu().contiguous().view(torch.uint8).numpy().tobytes()


def normal(shape, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def fenced(t):
    """A copy of t with NaN before and after it in memory, at t's alignment."""
    flat = torch.full((t.numel() + 2048,), float("nan"), dtype=t.dtype, device="cuda")
    inner = flat[1024:1024 + t.numel()].view(t.shape)
    inner.copy_(t)
    return inner


@pytest.mark.parametrize("n,topk,n_experts", [(1, 2, 16), (700, 3, 40), (40000, 2, 1024)])
def test_routing_stays_inside_its_buffers(gpu_lib, n, topk, n_experts):
    g = torch.Generator(device="cuda")
    g.manual_seed(n)
    ids = torch.randint(-1, n_experts, (n, topk), generator=g, device="cuda")
    ref = gpu_lib.kmeans_route(ids, n_experts)
    out = [like(t) for t in ref]
    ws = Guarded((gpu_lib.route_workspace(n, topk, n_experts).numel(),), torch.uint8, 0xFF)
    gpu_lib.kmeans_route(ids, n_experts, *[o.t for o in out], ws=ws.t)
    assert gpu_lib.kmeans_device_status(ws.t) == gpu_lib.KMEANS_OK
    assert ws.intact() and all(o.intact() for o in out)
    assert all(same(o.t, r) for o, r in zip(out, ref))


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("n,topk,d", [(3, 2, 64), (70, 3, 33), (500, 9, 1031), (300, 4, 2048)])
def test_row_movers_stay_inside_their_buffers(gpu_lib, n, topk, d, dtype):
    g = torch.Generator(device="cuda")
    g.manual_seed(d)
    ids = torch.randint(-1, 12, (n, topk), generator=g, device="cuda")
    offsets, _, rows = gpu_lib.kmeans_route(ids, 12)
    x, w = fenced(normal((n, d), dtype, 1)), torch.rand(n, topk, generator=g, device="cuda")
    ref = gpu_lib.kmeans_route_gather(x, rows, offsets)
    xs = like(ref)
    gpu_lib.kmeans_route_gather(x, rows, offsets, xs=xs.t)
    assert xs.intact() and same(xs.t, ref) and not torch.isnan(xs.t).any()
    ys = fenced(normal((n * topk, d), dtype, 2))
    ref = gpu_lib.kmeans_route_combine(ys, rows, offsets, weights=w, residual=x)
    y = like(ref)
    gpu_lib.kmeans_route_combine(ys, rows, offsets, weights=w, residual=x, y=y.t)
    assert y.intact() and same(y.t, ref) and not torch.isnan(y.t).any()
    ref = gpu_lib.kmeans_route_combine_grad(x, ys, rows, offsets, w)
    out = [like(t) for t in ref]
    gpu_lib.kmeans_route_combine_grad(x, ys, rows, offsets, w, dys=out[0].t, dweights=out[1].t)
    assert all(o.intact() and same(o.t, r) and not torch.isnan(o.t).any() for o, r in zip(out, ref))


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("m,n_experts,n,k", [(3, 1, 40, 72), (7, 5, 33, 51), (40, 9, 264, 136), (300, 1, 1000, 520),
                                             (333, 4, 515, 77), (900, 5, 520, 264), (2000, 3, 129, 1032)])
def test_products_stay_inside_their_buffers(gpu_lib, m, n_experts, n, k, dtype):
    r = np.random.RandomState(m)
    counts = r.multinomial(m - m // 10, np.full(n_experts, 1.0 / n_experts))
    offsets = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).cuda()
    x, w = fenced(normal((m, k), dtype, 1)), fenced(normal((n_experts, n, k), dtype, 2, k ** -0.5))
    bias, res = fenced(normal((n_experts, n), dtype, 3)), fenced(normal((m, n), dtype, 4))
    dy, pre = fenced(normal((m, n), dtype, 5)), fenced(normal((m, n), dtype, 6))
    args = dict(bias=bias, residual=res, offsets=offsets, activation="gelu")
    ref = gpu_lib.kmeans_linear(x, w, save_pre=True, **args)
    out = [like(t) for t in ref]
    ws = Guarded((gpu_lib.linear_workspace(gpu_lib.OP_LINEAR, m, n, k, n_experts).numel(),), torch.uint8, 0xFF)
    gpu_lib.kmeans_linear(x, w, y=out[0].t, pre=out[1].t, ws=ws.t, **args)
    assert gpu_lib.kmeans_device_status(ws.t) == gpu_lib.KMEANS_OK
    assert ws.intact() and all(o.intact() and same(o.t, r) and not torch.isnan(o.t).any() for o, r in zip(out, ref))
    ref = gpu_lib.kmeans_linear_grad(dy, x, w, pre=pre, offsets=offsets, activation="gelu")
    out = [like(t) for t in ref]
    ws = Guarded((gpu_lib.linear_workspace(gpu_lib.OP_LINEAR_GRAD, m, n, k, n_experts).numel(),), torch.uint8, 0xFF)
    gpu_lib.kmeans_linear_grad(dy, x, w, pre=pre, offsets=offsets, activation="gelu", dx=out[0].t, dw=out[1].t,
                               db=out[2].t, ws=ws.t)
    assert gpu_lib.kmeans_device_status(ws.t) == gpu_lib.KMEANS_OK
    assert ws.intact() and all(o.intact() and same(o.t, r) and not torch.isnan(o.t).any() for o, r in zip(out, ref))


def test_a_plan_with_rows_out_of_range_is_left_out(gpu_lib):
    n, topk, d = 50, 2, 40
    ids = torch.randint(0, 6, (n, topk), device="cuda")
    offsets, _, rows = gpu_lib.kmeans_route(ids, 6)
    x, ys, w = normal((n, d), torch.float32, 1), normal((n * topk, d), torch.float32, 2), torch.rand(n, topk, device="cuda")
    bad = rows.clone()
    bad[3, 1], bad[7, 0], bad[9, 1] = -4, n * topk, 2 ** 31 - 1
    xs = like(gpu_lib.kmeans_route_gather(x, rows, offsets))
    gpu_lib.kmeans_route_gather(x, bad, offsets, xs=xs.t)
    assert xs.intact()
    y = gpu_lib.kmeans_route_combine(ys, bad, offsets, weights=w)
    full = gpu_lib.kmeans_route_combine(ys, rows, offsets, weights=w)
    keep = torch.ones(n, dtype=torch.bool, device="cuda")
    keep[[3, 7, 9]] = False
    assert torch.equal(y[keep], full[keep])
    assert torch.allclose(y[7], w[7, 1] * ys[rows[7, 1].long()], rtol=1e-6)
    dys = like(ys)
    _, dw = gpu_lib.kmeans_route_combine_grad(x, ys, bad, offsets, w, dys=dys.t)
    assert dys.intact() and dw[3, 1] == 0 and dw[7, 0] == 0 and dw[9, 1] == 0


def test_each_call_sees_what_was_written_just_before_it(gpu_lib):
    """The first kernel of a call may be scheduled while the caller's last one
    still runs; it must wait for it."""
    n, d, E = 4096, 512, 8
    ids = torch.randint(0, E, (n, 2), device="cuda")
    offsets, _, rows = gpu_lib.kmeans_route(ids, E)
    w1 = normal((E, d, d), torch.bfloat16, 1, d ** -0.5)
    wts = torch.rand(n, 2, device="cuda")
    few = torch.tensor([0, 1, 2, 3, 4, 4, 4, 4, 4], dtype=torch.int32, device="cuda")
    big = normal((4096, 4096), torch.float32, 9)

    def chain(x, fresh):
        out = []
        for call in (lambda t: gpu_lib.kmeans_route_gather(t, rows, offsets),
                     lambda t: gpu_lib.kmeans_route_combine(t.repeat(2, 1), rows, offsets, weights=wts),
                     lambda t: gpu_lib.kmeans_linear(t.repeat(2, 1), w1, offsets=offsets)[0],
                     lambda t: gpu_lib.kmeans_linear(t[:4].clone(), w1, offsets=few)[0],
                     lambda t: gpu_lib.kmeans_linear_grad(t.repeat(2, 1), t.repeat(2, 1), w1, offsets=offsets)[1]):
            if fresh:
                torch.cuda.synchronize()
                out.append(call(x))
                torch.cuda.synchronize()
            else:
                t = torch.zeros_like(x)
                (big @ big).mean()  # keeps the stream busy
                t.copy_(x)
                out.append(call(t))
        return out

    for seed in range(3):
        x = normal((n, d), torch.bfloat16, seed)
        for a, b in zip(chain(x, False), chain(x, True)):
            assert torch.equal(a, b)

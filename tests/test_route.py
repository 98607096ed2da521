"""Expert routing on the GPU against a plain implementation in float64.

Bounds, fixed before any run: moved rows are exact; a sum of T terms in
float32 is within (T + 2) 2^-24 of the sum of its terms' magnitudes, and a
result kept in b significant bits within 2^-b of itself (float16 also within
2^-25, half its smallest step).
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

BITS = {torch.float32: 24, torch.float16: 11, torch.bfloat16: 8}
TINY = {torch.float32: 0.0, torch.float16: 2.0 ** -25, torch.bfloat16: 0.0}
DTYPES = [torch.float32, torch.float16, torch.bfloat16]


def plain_route(ids, n_experts):
    """(offsets, order, rows) by definition: a stable sort, dropped slots last."""
    flat = ids.reshape(-1).astype(np.int64)
    key = np.where((flat < 0) | (flat >= n_experts), n_experts, flat)
    order = np.argsort(key, kind="stable")
    rows = np.empty_like(order)
    rows[order] = np.arange(order.size)
    offsets = np.array([(key < e).sum() for e in range(n_experts + 1)])
    return offsets, order, rows.reshape(ids.shape)


def draw_ids(n, topk, n_experts, drop, seed, dtype=np.int64):
    r = np.random.RandomState(seed)
    ids = r.randint(0, n_experts, size=(n, topk))
    ids[r.rand(n, topk) < drop] = -1 - r.randint(0, 3)
    return ids.astype(dtype)


def plan(km, ids, n_experts):
    out = km.kmeans_route(torch.from_numpy(ids).cuda(), n_experts)
    return out


def normal(shape, dtype, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def within(got, want, size, terms, dtype):
    """`size`: the sum of the terms' magnitudes."""
    bound = (terms + 2) * 2.0 ** -24 * size + 2.0 ** -BITS[dtype] * want.abs() * 1.01 + TINY[dtype]
    off = (got.double() - want).abs()
    assert bool((off <= bound).all()), f"off by {(off - bound).max().item():.3e} more than the bound"


@pytest.mark.parametrize("id_dtype", [np.int32, np.int64])
@pytest.mark.parametrize("n,topk,n_experts,drop", [
    (0, 2, 4, 0.0), (1, 1, 1, 0.0), (1, 1, 3, 1.0), (31, 1, 2, 0.3), (33, 3, 7, 0.1), (257, 8, 128, 0.0),
    (4097, 1, 1000, 0.02), (5000, 4, 4096, 0.5), (70001, 2, 64, 0.05), (300000, 1, 1024, 0.0), (513, 32, 40, 1.0),
    (9, 0, 5, 0.0),
])
def test_slots_are_sorted_by_expert_in_slot_order(gpu_lib, n, topk, n_experts, drop, id_dtype):
    ids = draw_ids(n, topk, n_experts, drop, seed=n + topk + n_experts, dtype=id_dtype)
    ws = gpu_lib.route_workspace(n, topk, n_experts)
    got = gpu_lib.kmeans_route(torch.from_numpy(ids).cuda(), n_experts, ws=ws)
    assert gpu_lib.kmeans_device_status(ws) == gpu_lib.KMEANS_OK
    for a, b in zip(got, plain_route(ids, n_experts)):
        assert a.dtype == torch.int32
        assert np.array_equal(a.cpu().numpy(), b)


@pytest.mark.parametrize("n", [1000, 40000])
def test_one_popular_expert(gpu_lib, n):
    ids = np.full((n, 2), 5, dtype=np.int64)
    ids[n // 2, 1] = 4
    for a, b in zip(plan(gpu_lib, ids, 9), plain_route(ids, 9)):
        assert np.array_equal(a.cpu().numpy(), b)


@pytest.mark.parametrize("bad", [6, 2 ** 31 - 1, 2 ** 40])
def test_an_id_past_the_experts_is_dropped_and_reported(gpu_lib, bad):
    ids = draw_ids(500, 2, 6, 0.1, seed=3)
    ids[123, 1] = bad
    ws = gpu_lib.route_workspace(500, 2, 6)
    got = gpu_lib.kmeans_route(torch.from_numpy(ids).cuda(), 6, ws=ws)
    assert gpu_lib.kmeans_device_status(ws) == gpu_lib.KMEANS_ERR_DEVICE_LABEL
    for a, b in zip(got, plain_route(ids, 6)):
        assert np.array_equal(a.cpu().numpy(), b)
    ids[123, 1] = -7  # the next call on the workspace starts clean
    gpu_lib.kmeans_route(torch.from_numpy(ids).cuda(), 6, ws=ws)
    assert gpu_lib.kmeans_device_status(ws) == gpu_lib.KMEANS_OK


SHAPES = [(1, 1, 1, 1, 0.0), (3, 2, 4, 8, 1.0), (5, 3, 7, 33, 0.2), (64, 9, 16, 512, 0.1), (257, 2, 5, 64, 0.0),
          (1000, 8, 128, 1031, 0.05), (130, 32, 40, 2048, 0.3), (17, 4, 64, 8200, 0.0), (2, 0, 3, 16, 0.0)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,topk,n_experts,d,drop", SHAPES)
def test_gather_copies_each_token_to_its_rows(gpu_lib, n, topk, n_experts, d, drop, dtype):
    ids = draw_ids(n, topk, n_experts, drop, seed=d)
    offsets, order, rows = plan(gpu_lib, ids, n_experts)
    x = normal((n, d), dtype, 1)
    xs = gpu_lib.kmeans_route_gather(x, rows, offsets, xs=torch.full((n * topk, d), 7.0, dtype=dtype, device="cuda"))
    kept = int(offsets[-1])
    want = torch.zeros_like(xs)
    want[:kept] = x[order[:kept].long() // max(topk, 1)]
    assert torch.equal(xs, want)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,topk,n_experts,d,drop", SHAPES)
@pytest.mark.parametrize("weighted,residual", [(True, True), (False, False)])
def test_combine_adds_the_weighted_rows(gpu_lib, n, topk, n_experts, d, drop, dtype, weighted, residual):
    ids = draw_ids(n, topk, n_experts, drop, seed=d + 1)
    offsets, _, rows = plan(gpu_lib, ids, n_experts)
    kept = rows < offsets[-1]
    ys = normal((n * topk, d), dtype, 2)
    w = torch.rand(n, topk, device="cuda")
    res = normal((n, d), dtype, 3) if residual else None
    ys[int(offsets[-1]):] = float("nan")  # rows of dropped choices hold anything
    w[~kept] = float("inf")
    y = gpu_lib.kmeans_route_combine(ys, rows, offsets, weights=w if weighted else None, residual=res)
    part = torch.zeros(n, topk, d, dtype=torch.float64, device="cuda")
    part[kept] = ys[rows[kept].long()].double() * (w[kept].double()[:, None] if weighted else 1.0)
    want, size = part.sum(1), part.abs().sum(1)
    if residual:
        want, size = want + res.double(), size + res.double().abs()
    within(y, want, size, topk + 1, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,topk,n_experts,d,drop", SHAPES)
def test_gradient_of_the_combine(gpu_lib, n, topk, n_experts, d, drop, dtype):
    ids = draw_ids(n, topk, n_experts, drop, seed=d + 2)
    offsets, _, rows = plan(gpu_lib, ids, n_experts)
    kept = rows < offsets[-1]
    ys, dy = normal((n * topk, d), dtype, 4), normal((n, d), dtype, 5)
    w = torch.rand(n, topk, device="cuda")
    ys[int(offsets[-1]):] = float("nan")
    dys = torch.full_like(ys, 7.0)
    dys, dw = gpu_lib.kmeans_route_combine_grad(dy, ys, rows, offsets, torch.where(kept, w, float("nan")), dys=dys)
    # by the formula
    want = torch.zeros(n * topk, d, dtype=torch.float64, device="cuda")
    t, j = kept.nonzero(as_tuple=True)
    want[rows[t, j].long()] = w[t, j].double()[:, None] * dy[t].double()
    within(dys, want, want.abs(), 1, dtype)
    prod = dy[t].double() * ys[rows[t, j].long()].double()
    want_w, size = torch.zeros(n, topk, dtype=torch.float64, device="cuda"), torch.zeros(n, topk, dtype=torch.float64,
                                                                                         device="cuda")
    want_w[t, j], size[t, j] = prod.sum(1), prod.abs().sum(1)
    within(dw, want_w, size, d, torch.float32)


def test_gradients_agree_with_differences(gpu_lib):
    # y is linear in ys and in the weights, so a difference over a step h is
    # off by y's own float32 rounding alone: 8 2^-24 |y| / h in each element
    n, topk, n_experts, d, h = 20, 3, 6, 24, 0.5
    ids = draw_ids(n, topk, n_experts, 0.2, seed=8)
    offsets, _, rows = plan(gpu_lib, ids, n_experts)
    x, ys, dy = (normal(s, torch.float32, i) for i, s in enumerate([(n, d), (n * topk, d), (n, d)]))
    w = torch.rand(n, topk, device="cuda")
    dys, dw = gpu_lib.kmeans_route_combine_grad(dy, ys, rows, offsets, w)
    dx = gpu_lib.kmeans_route_combine(dys, rows, offsets)  # the gather's gradient

    def loss(ys, w):
        return (gpu_lib.kmeans_route_combine(ys, rows, offsets, weights=w).double() * dy.double()).sum().item()

    def gather_loss(x):
        return (gpu_lib.kmeans_route_gather(x, rows, offsets).double() * dys.double()).sum().item()

    bound = 64 * d * 2.0 ** -24 * 20 / h
    r = np.random.RandomState(0)
    for _ in range(10):
        i, c, t, j = r.randint(n * topk), r.randint(d), r.randint(n), r.randint(topk)
        for value, grad, at, f in ((ys, dys, (i, c), lambda v: loss(v, w)), (w, dw, (t, j), lambda v: loss(ys, v)),
                                   (x, dx, (t, c), gather_loss)):
            up, down = value.clone(), value.clone()
            up[at] += h
            down[at] -= h
            step = (up[at] - down[at]).item()
            assert abs((f(up) - f(down)) / step - grad[at].item()) <= bound


@pytest.mark.parametrize("dtype", DTYPES)
def test_strided_rows_and_other_streams(gpu_lib, dtype):
    n, topk, n_experts, d = 100, 2, 8, 40
    ids = draw_ids(n, topk, n_experts, 0.1, seed=4)
    side = torch.cuda.Stream()
    for pitch, first in ((64, 8), (57, 3)):
        wide = normal((n, pitch), dtype, 6)
        x = wide[:, first:first + d]
        offsets, order, rows = plan(gpu_lib, ids, n_experts)
        ref = gpu_lib.kmeans_route_gather(x.contiguous(), rows, offsets)
        w = torch.rand(n, topk, device="cuda")
        back = gpu_lib.kmeans_route_combine(ref, rows, offsets, weights=w, residual=x.contiguous())
        grads = gpu_lib.kmeans_route_combine_grad(x.contiguous(), ref, rows, offsets, w)
        torch.cuda.synchronize()
        got = gpu_lib.kmeans_route_gather(x, rows, offsets, xs=torch.empty_like(ref), stream=side)
        side.synchronize()
        assert torch.equal(got, ref)
        assert torch.equal(gpu_lib.kmeans_route_combine(ref, rows, offsets, weights=w, residual=x), back)
        for a, b in zip(gpu_lib.kmeans_route_combine_grad(x, ref, rows, offsets, w), grads):
            assert torch.equal(a, b)


def test_residual_in_place_and_whole_chain_in_a_graph(gpu_lib):
    n, topk, n_experts, d = 65, 2, 8, 128
    ids = torch.from_numpy(draw_ids(n, topk, n_experts, 0.1, seed=5)).cuda()
    x = normal((n, d), torch.bfloat16, 7)
    w = torch.rand(n, topk, device="cuda")
    ws = gpu_lib.route_workspace(n, topk, n_experts)
    offsets, order, rows = gpu_lib.kmeans_route(ids, n_experts, ws=ws)
    xs = gpu_lib.kmeans_route_gather(x, rows, offsets)
    want = gpu_lib.kmeans_route_combine(xs, rows, offsets, weights=w, residual=x)
    y = x.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gpu_lib.kmeans_route(ids, n_experts, offsets=offsets, order=order, rows=rows, ws=ws)
        gpu_lib.kmeans_route_gather(x, rows, offsets, xs=xs)
        gpu_lib.kmeans_route_combine(xs, rows, offsets, weights=w, residual=y, y=y)
    for t in (offsets, order, rows):
        t.fill_(-1)
    xs.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want)


def test_more_than_two_to_the_31_elements(gpu_lib):
    n, topk, n_experts, d = 33000, 8, 16, 8192
    ids = draw_ids(n, topk, n_experts, 0.01, seed=6)
    offsets, order, rows = plan(gpu_lib, ids, n_experts)
    assert n * topk * d > 2 ** 31
    x = normal((n, d), torch.bfloat16, 8)
    xs = gpu_lib.kmeans_route_gather(x, rows, offsets)
    kept = int(offsets[-1])
    at = torch.tensor([0, 1, kept // 2, kept - 2, kept - 1], device="cuda")
    assert torch.equal(xs[at], x[order[at].long() // topk])
    assert not xs[kept:].any()
    w = torch.rand(n, topk, device="cuda")
    y = gpu_lib.kmeans_route_combine(xs, rows, offsets, weights=w)
    last = torch.arange(n - 50, n, device="cuda")
    total = (w * (rows < kept)).double().sum(1)[last]
    want = total[:, None] * x[last].double()
    within(y[last], want, want.abs() * topk, topk, torch.bfloat16)
    dys, dw = gpu_lib.kmeans_route_combine_grad(x, xs, rows, offsets, w)
    r = rows[last].long()
    ref = w[last].double()[:, :, None] * x[last].double()[:, None, :] * (r < kept)[:, :, None]
    within(dys[r], ref, ref.abs(), 1, torch.bfloat16)

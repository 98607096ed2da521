"""Products over long contractions, all terms of one sign: what the tensor cores
cut off may not add up over the contraction.

Bounds, fixed before any run.  An accumulator takes 32768 terms at most, 16 to an
addition, and each of those 2048 additions cuts off up to 2^-23 of the sum: 2^-12
of it.  The chunks' sums meet in float32, within K / 32768 additions of 2^-24, and
a result in b bits is within 2^-b of itself.  The bound does not grow with K but
by those few 2^-24."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

BITS = {torch.float16: 11, torch.bfloat16: 8}


def positive(shape, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    out = torch.empty(shape, dtype=dtype, device="cuda")
    for i in range(0, shape[0], 1024):  # (the float32 values of 20 GB would not be small)
        part = out[i:i + 1024]
        part.copy_((torch.rand(part.shape, generator=g, device="cuda") * 0.5 + 0.5) * scale)
    return out


def exact(a, b):
    """a b^T over the last dimension."""
    return sum(a[:, i:i + 65536].double() @ b[:, i:i + 65536].double().t() for i in range(0, a.shape[1], 65536))


def close(got, want, k, dtype, extra=0.0):
    bound = (2.0 ** -12 + (k / 32768 + 20) * 2.0 ** -24 + 2.0 ** -BITS[dtype]) * want.abs() + extra
    off = (got.double() - want).abs()
    assert bool((off <= bound).all()), f"off by {((off - bound) / want.abs()).max().item():.2e} more than the bound"


LONG = [32768 + 8, 65536, 131072, 262144 + 40, 1 << 20]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("k", LONG)
@pytest.mark.parametrize("m,n", [(9, 40), (300, 72)])
def test_forward(gpu_lib, m, n, k, dtype):
    x, w = positive((m, k), dtype, 1), positive((n, k), dtype, 2, 2.0 ** -7)
    ws = gpu_lib.linear_workspace(gpu_lib.OP_LINEAR, m, n, k)
    ws.fill_(0xFF)
    y, _ = gpu_lib.kmeans_linear(x, w, ws=ws)
    assert gpu_lib.kmeans_device_status(ws) == gpu_lib.KMEANS_OK
    close(y, exact(x, w), k, dtype)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("n", LONG)
@pytest.mark.parametrize("m,k", [(9, 40), (300, 72)])
def test_gradient_of_the_rows(gpu_lib, m, n, k, dtype):
    dy, w = positive((m, n), dtype, 1), positive((n, k), dtype, 2, 2.0 ** -7)
    x = positive((m, k), dtype, 3)
    ws = gpu_lib.linear_workspace(gpu_lib.OP_LINEAR_GRAD, m, n, k)
    ws.fill_(0xFF)
    dx, dw, _ = gpu_lib.kmeans_linear_grad(dy, x, w, need_db=False, ws=ws)
    assert gpu_lib.kmeans_device_status(ws) == gpu_lib.KMEANS_OK
    close(dx, exact(dy, w.t().contiguous()), n, dtype)
    close(dw, dy.t().double() @ x.double(), m, dtype)


def test_experts_with_everything(gpu_lib):
    """Several units per pair, ragged experts and dropped rows, bias, activation,
    residual and the kept values; outputs on and off 16 bytes."""
    k, counts, dropped = 70000, [700, 0, 1, 333, 260], 9
    m = sum(counts) + dropped
    edges = [0]
    for c in counts:
        edges.append(edges[-1] + c)
    offsets = torch.tensor(edges, dtype=torch.int32, device="cuda")
    x = positive((m, k), torch.float16, 1)
    for n in (1032, 515):
        w = positive((5 * n, k), torch.float16, 2, 2.0 ** -10).view(5, n, k)
        bias, res = positive((5, n), torch.float16, 3, 8.0), positive((m, n), torch.float16, 4, 64.0)
        ws = gpu_lib.linear_workspace(gpu_lib.OP_LINEAR, m, n, k, 5)
        ws.fill_(0xFF)
        y, pre = gpu_lib.kmeans_linear(x, w, bias=bias, residual=res, offsets=offsets, activation="relu", save_pre=True,
                                       ws=ws)
        assert gpu_lib.kmeans_device_status(ws) == gpu_lib.KMEANS_OK
        for e in range(5):
            a, b = edges[e], edges[e + 1]
            z = exact(x[a:b], w[e]) + bias[e].double()
            close(pre[a:b], z, k, torch.float16)
            close(y[a:b], z + res[a:b].double(), k, torch.float16)
        assert not y[edges[-1]:].any() and not pre[edges[-1]:].any()
        again, _ = gpu_lib.kmeans_linear(x, w, bias=bias, residual=res, offsets=offsets, activation="relu", ws=ws)
        assert torch.equal(again, y)


@pytest.mark.parametrize("m,n,k", [(4, 9728, 1 << 20), (3, 200, 1 << 19), (8, 40, (1 << 21) + 64), (1, 33, 262144 + 5)])
def test_few_rows(gpu_lib, m, n, k):
    """9728 features give every block a unit of its own, so that nothing but the
    length asks for a split of the contraction."""
    torch.cuda.empty_cache()
    x, w = positive((m, k), torch.float16, 1), positive((n, k), torch.float16, 2, 2.0 ** -8)
    y, _ = gpu_lib.kmeans_linear(x, w)
    some = slice(0, 64)
    close(y[:, some], exact(x, w[some]), k, torch.float16)
    close(y[:, n - 20:], exact(x, w[n - 20:]), k, torch.float16)
    del w
    torch.cuda.empty_cache()


@pytest.mark.parametrize("m,experts,need_dw", [(1 << 27, 1, True), (1 << 27, 1, False), (1 << 25, 1024, True)])
def test_bias_gradient_of_many_equal_rows(gpu_lib, m, experts, need_dw):
    """Alone, and beside the weight gradient (all rows with one of 1024 experts).
    A tile's sum is of 128 rows, each within 2^-24 per addition; the tiles' sums
    meet with their errors, the last rounding is float16's 2^-11."""
    torch.cuda.empty_cache()
    dy = torch.full((m, 8), 0.0004, dtype=torch.float16, device="cuda")
    x = torch.zeros(m, 8, dtype=torch.float16, device="cuda")
    w = torch.zeros((experts, 8, 8) if experts > 1 else (8, 8), dtype=torch.float16, device="cuda")
    offsets = None
    if experts > 1:
        offsets = torch.zeros(experts + 1, dtype=torch.int32, device="cuda")
        offsets[8:] = m
    _, dw, db = gpu_lib.kmeans_linear_grad(dy, x, w, offsets=offsets, need_dx=False, need_dw=need_dw)
    want = m * dy[0, 0].double()
    got = (db[7] if experts > 1 else db).double()
    assert bool(((got - want).abs() <= (2.0 ** -11 + 130 * 2.0 ** -24) * want).all()), ((got - want) / want).tolist()
    if experts > 1:
        assert not db[:7].any() and not db[8:].any()
    dy[m // 2, 3] = float("inf")  # an infinite sum stays one
    _, _, db = gpu_lib.kmeans_linear_grad(dy, x, w, offsets=offsets, need_dx=False, need_dw=need_dw)
    assert (db[7] if experts > 1 else db)[3].item() == float("inf") and int(torch.isfinite(db).logical_not().sum()) == 1
    del x, dy
    torch.cuda.empty_cache()


@pytest.mark.parametrize("m", [40, 700])
def test_a_starved_long_contraction_reports_a_timeout(gpu_lib, monkeypatch, m):
    k = 70000
    x, w = positive((m, k), torch.bfloat16, 1), positive((264, k), torch.bfloat16, 2, 2.0 ** -8)
    ws = gpu_lib.linear_workspace(gpu_lib.OP_LINEAR, m, 264, k)
    ref = gpu_lib.kmeans_linear(x, w)[0]
    monkeypatch.setenv("KMEANS_GB300_TEST_STARVE_PIPELINE", "1")
    gpu_lib.kmeans_linear(x, w, ws=ws)
    assert gpu_lib.kmeans_device_status(ws) == gpu_lib.KMEANS_ERR_DEVICE_TIMEOUT
    monkeypatch.delenv("KMEANS_GB300_TEST_STARVE_PIPELINE")
    assert torch.equal(gpu_lib.kmeans_linear(x, w, ws=ws)[0], ref)
    assert gpu_lib.kmeans_device_status(ws) == gpu_lib.KMEANS_OK

"""The products at the ends of their sizes: refusals on the host, and on the GPU
rows that reach up to the limit, exact on small whole numbers."""
import ctypes

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def km():
    from distance_argmin_gb300 import build as b
    b.build()
    import distance_argmin_gb300 as km
    km.load()
    return km


def test_sizes_past_the_limits_are_refused_on_the_host(km):
    lib, top = km.load(), km.LINEAR_MAX_SIZE
    assert top == 2 ** 31 - 256
    fake, ws = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x100000)  # never dereferenced: validation fails first
    for m, n, k, experts in ((top + 1, 8, 8, 1), (8, top + 1, 8, 1), (8, 8, top + 1, 1), (2 ** 31 - 1, 8, 8, 1),
                             (top, 2049, 8, 1), (top, 8, 2049, 1), (8, top // 1024, 2 ** 22, 1024), (top, top, top, 1)):
        for grad in (0, 1):
            assert lib.kmeans_linear_workspace_bytes(grad, m, n, k, experts) == 0
        forward = lib.kmeans_linear(fake, k, fake, None, None, 0, km.BF16, 0, fake, m, n, k, experts, fake, None, ws,
                                    2 ** 63, None)
        grads = lib.kmeans_linear_grad(fake, n, fake, k, fake, None, km.BF16, 0, fake, m, n, k, experts, fake, fake,
                                       fake, ws, 2 ** 63, None)
        assert forward == grads == km.KMEANS_ERR_INVALID_ARG
    # the largest that are taken need what their matrices do, not less
    for m, n, k in ((top, 8, 8), (8, top, 8), (8, 8, top), (top, 2048, 8), (top, 8, 2048)):
        need = lib.kmeans_linear_workspace_bytes(1, m, n, k, 1)
        assert need >= 2 * m * n + 2 * m * k and need < 2 ** 50


@pytest.mark.gpu
@pytest.mark.parametrize("split", [None, 2 ** 31 - 40000])
def test_rows_up_to_the_limit(gpu_lib, split):
    """The rows' chunks and tiles end at 2^31 - 256.  Values -1, 0 and 1 in the
    first and the last rows, zeros between: every sum is a whole number that 16
    bits hold."""
    m, d, ends = gpu_lib.LINEAR_MAX_SIZE, 8, 70000
    torch.cuda.empty_cache()
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    whole = lambda *shape: torch.randint(-1, 2, shape, generator=g, device="cuda").half()
    x, dy = torch.zeros(m, d, dtype=torch.float16, device="cuda"), torch.zeros(m, d, dtype=torch.float16, device="cuda")
    for t in (x, dy):
        t[:ends], t[-ends:] = whole(ends, d), whole(ends, d)
    experts = 1 if split is None else 2
    w = whole(experts, d, d)
    offsets = None if split is None else torch.tensor([0, split, m], dtype=torch.int32, device="cuda")
    ws = gpu_lib.linear_workspace(gpu_lib.OP_LINEAR_GRAD, m, d, d, experts)
    _, dw, db = gpu_lib.kmeans_linear_grad(dy, x, w, offsets=offsets, need_dx=False, ws=ws)
    assert gpu_lib.kmeans_device_status(ws) == gpu_lib.KMEANS_OK
    edges = [0, m] if split is None else [0, split, m]
    for e in range(experts):
        parts = [(max(a, edges[e]), min(b, edges[e + 1])) for a, b in ((0, ends), (m - ends, m))]
        want_w = sum(dy[a:b].double().t() @ x[a:b].double() for a, b in parts if a < b)
        want_b = sum(dy[a:b].double().sum(0) for a, b in parts if a < b)
        assert torch.equal(dw[e].double(), want_w) and torch.equal(db[e].double(), want_b)
    del ws
    wf = gpu_lib.linear_workspace(gpu_lib.OP_LINEAR, m, d, d, experts)
    y, _ = gpu_lib.kmeans_linear(x, w, offsets=offsets, ws=wf)
    assert gpu_lib.kmeans_device_status(wf) == gpu_lib.KMEANS_OK
    last = (m - 30000, m)  # one expert's
    assert torch.equal(y[slice(*last)].double(), x[slice(*last)].double() @ w[-1].double().t())
    assert torch.equal(y[:ends].double(), x[:ends].double() @ w[0].double().t())
    del y, wf, x, dy
    torch.cuda.empty_cache()


@pytest.mark.gpu
@pytest.mark.parametrize("k", [2 ** 30 + 8, 2 ** 30 + 1])
def test_a_row_of_more_than_two_to_the_31_bytes(gpu_lib, k):
    """As it lies, and brought to 16 bytes first: terms at both ends and between,
    zeros elsewhere."""
    torch.cuda.empty_cache()
    x, w = torch.zeros(1, k, dtype=torch.float16, device="cuda"), torch.zeros(1, k, dtype=torch.float16, device="cuda")
    at = torch.tensor([0, 7, 12345, 2 ** 21 + 3, 2 ** 29 + 5, 2 ** 30 - 1, k - 1], device="cuda")
    x[0, at] = torch.tensor([1, 2, 4, 8, 16, 32, 64], dtype=torch.float16, device="cuda")
    w[0, at] = torch.tensor([3, -1, 5, 7, -2, 1, 3], dtype=torch.float16, device="cuda")
    ws = gpu_lib.linear_workspace(gpu_lib.OP_LINEAR, 1, 1, k)
    y, _ = gpu_lib.kmeans_linear(x, w, ws=ws)
    assert gpu_lib.kmeans_device_status(ws) == gpu_lib.KMEANS_OK
    assert y.item() == (x[0, at] * w[0, at]).double().sum().item()
    del ws
    dy = torch.full((1, 1), 3.0, dtype=torch.float16, device="cuda")
    ws = gpu_lib.linear_workspace(gpu_lib.OP_LINEAR_GRAD, 1, 1, k)
    dx, dw, db = gpu_lib.kmeans_linear_grad(dy, x, w, ws=ws)
    assert gpu_lib.kmeans_device_status(ws) == gpu_lib.KMEANS_OK
    assert torch.equal(dx[0, at], 3 * w[0, at]) and torch.equal(dw[0, at], 3 * x[0, at]) and db.item() == 3
    assert int(dx.count_nonzero()) == int(dw.count_nonzero()) == at.numel()
    del x, w, dx, dw, ws
    torch.cuda.empty_cache()

"""The status word of the products: whatever a workspace held before, a call
reports its own waits and nobody else's."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from test_linear import normal  # noqa: E402


def product_first(km, m, n, k, ws, seed=0):
    """A call whose only kernel is the product (rows on 16 bytes)."""
    x, w = normal((m, k), torch.bfloat16, seed), normal((n, k), torch.bfloat16, seed + 1)
    return km.kmeans_linear(x, w, ws=ws)[0], x, w


@pytest.mark.parametrize("m,n", [(40, 64), (3000, 1536)])
@pytest.mark.parametrize("left", [0x00, 0x01, 0xFF])
def test_what_the_workspace_held_is_not_taken_for_an_error(gpu_lib, m, n, left):
    ws = gpu_lib.linear_workspace(gpu_lib.OP_LINEAR, m, n, 512)
    ref = product_first(gpu_lib, m, n, 512, None)[0]
    for _ in range(20):
        ws.fill_(left)
        y = product_first(gpu_lib, m, n, 512, ws)[0]
        assert gpu_lib.kmeans_device_status(ws) == gpu_lib.KMEANS_OK
        assert torch.equal(y, ref)


def test_a_timeout_is_reported_once_by_the_call_that_had_it(gpu_lib, monkeypatch):
    big = (3000, 1536, 512)  # every pair of SMs has units
    ws = gpu_lib.linear_workspace(gpu_lib.OP_LINEAR_GRAD, *big)
    ref, x, w = product_first(gpu_lib, *big, None)
    small, xs, w2 = product_first(gpu_lib, 40, 64, 512, None)
    dy = normal((3000, 1536), torch.bfloat16, 7)
    grad = lambda: gpu_lib.kmeans_linear_grad(dy, x, w, need_db=False, ws=ws)  # rows first, weights second
    dx, dw, _ = grad()
    assert gpu_lib.kmeans_device_status(ws) == gpu_lib.KMEANS_OK
    for starved in (lambda: gpu_lib.kmeans_linear(x, w, ws=ws), grad):
        monkeypatch.setenv("KMEANS_GB300_TEST_STARVE_PIPELINE", "1")
        starved()
        assert gpu_lib.kmeans_device_status(ws) == gpu_lib.KMEANS_ERR_DEVICE_TIMEOUT
        monkeypatch.delenv("KMEANS_GB300_TEST_STARVE_PIPELINE")
        # a call on one pair, while the other pairs' words still hold the error
        assert torch.equal(gpu_lib.kmeans_linear(xs, w2, ws=ws)[0], small)
        assert gpu_lib.kmeans_device_status(ws) == gpu_lib.KMEANS_OK
        assert torch.equal(gpu_lib.kmeans_linear(x, w, ws=ws)[0], ref)
        assert gpu_lib.kmeans_device_status(ws) == gpu_lib.KMEANS_OK
        got = grad()
        assert gpu_lib.kmeans_device_status(ws) == gpu_lib.KMEANS_OK
        assert torch.equal(got[0], dx) and torch.equal(got[1], dw)
        # other operators on the same memory
        ids = torch.randint(0, 6, (100, 2), device="cuda")
        gpu_lib.kmeans_route(ids, 6, ws=ws)
        assert gpu_lib.kmeans_device_status(ws) == gpu_lib.KMEANS_OK
        ids[3, 1] = 6
        gpu_lib.kmeans_route(ids, 6, ws=ws)
        assert gpu_lib.kmeans_device_status(ws) == gpu_lib.KMEANS_ERR_DEVICE_LABEL


@pytest.mark.parametrize("m", [0, 64])
def test_a_gradient_of_nothing_leaves_a_clean_status(gpu_lib, m):
    x, w, dy = (normal(s, torch.float16, i) for i, s in enumerate([(m, 16), (24, 16), (m, 24)]))
    ws = gpu_lib.linear_workspace(gpu_lib.OP_LINEAR_GRAD, m, 24, 16)
    ws.fill_(1)
    out = gpu_lib.kmeans_linear_grad(dy, x, w, need_dx=False, need_dw=False, need_db=False, ws=ws)
    assert out == (None, None, None)
    assert gpu_lib.kmeans_device_status(ws) == gpu_lib.KMEANS_OK

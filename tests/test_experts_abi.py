"""Host-side checks of the expert routing and product entry points: argument
validation before anything touches the GPU, and workspace sizes.  No kernel
runs here (no GPU needed)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def km():
    from distance_argmin_gb300 import build as b
    b.build()
    import distance_argmin_gb300 as km
    km.load()
    return km


def _lib(km):
    return km.load()


FAKE = ctypes.c_void_p(0x10000)      # never dereferenced: validation fails first
FAKE_WS = ctypes.c_void_p(0x100000)  # 256-byte aligned


def test_expert_entry_points_validate_on_the_host(km):
    lib = _lib(km)
    F, W = FAKE, FAKE_WS
    BAD, NO, OK = km.KMEANS_ERR_INVALID_ARG, km.KMEANS_ERR_UNSUPPORTED, km.KMEANS_OK
    odd = ctypes.c_void_p(0x10001)
    assert km.ROUTE_MAX_EXPERTS == 4096 and km.LINEAR_MAX_EXPERTS == 1024  # mirrored defines
    assert lib.kmeans_route_workspace_bytes(100, 2, 8) >= 256
    for sizes in ((-1, 2, 8), (2 ** 30, 2, 8), (10, 33, 8), (10, 2, 0), (10, 2, 4097)):
        assert lib.kmeans_route_workspace_bytes(*sizes) == 0
    route = lambda ids=F, b=8, n=10, topk=2, E=8, off=F, order=F, rows=F, ws=W, wsb=256: \
        lib.kmeans_route(ids, b, n, topk, E, off, order, rows, ws, wsb, None)
    assert route(ids=None) == BAD and route(b=2) == BAD and route(off=None) == BAD and route(rows=None) == BAD
    assert route(ids=ctypes.c_void_p(0x10004)) == BAD and route(order=odd) == BAD
    assert route(n=2 ** 30) == BAD and route(n=-1) == BAD and route(E=0) == BAD
    assert route(topk=33) == NO and route(E=4097) == NO
    assert route(wsb=255) == km.KMEANS_ERR_WORKSPACE and route(ws=odd) == km.KMEANS_ERR_WORKSPACE
    gather = lambda x=F, ldx=16, dt=1, rows=F, off=F, n=10, topk=2, E=8, d=16, xs=F: \
        lib.kmeans_route_gather(x, ldx, dt, rows, off, n, topk, E, d, xs, None)
    assert gather(x=None) == BAD and gather(ldx=15) == BAD and gather(dt=3) == BAD and gather(xs=odd) == BAD
    assert gather(rows=None) == BAD and gather(off=odd) == BAD and gather(topk=40) == NO and gather(d=2 ** 24) == NO
    assert gather(n=0, x=None, rows=None, off=None, xs=None) == OK and gather(d=0) == OK  # nothing enqueued
    combine = lambda ys=F, dt=2, w=None, res=None, ldr=0, rows=F, off=F, n=10, topk=2, E=8, d=16, y=F: \
        lib.kmeans_route_combine(ys, dt, w, res, ldr, rows, off, n, topk, E, d, y, None)
    assert combine(ys=None) == BAD and combine(y=None) == BAD and combine(res=F, ldr=15) == BAD
    assert combine(w=ctypes.c_void_p(0x10002)) == BAD and combine(off=None) == BAD and combine(n=0) == OK
    cgrad = lambda dy=F, ld=16, ys=F, dt=0, w=F, rows=F, off=F, n=10, topk=2, E=8, d=16, dys=F, dw=F: \
        lib.kmeans_route_combine_grad(dy, ld, ys, dt, w, rows, off, n, topk, E, d, dys, dw, None)
    assert cgrad(w=None) == BAD and cgrad(dw=None) == BAD and cgrad(dys=None) == BAD and cgrad(ld=8) == BAD
    assert cgrad(dy=ctypes.c_void_p(0x10002)) == BAD and cgrad(topk=0) == OK

    need = lib.kmeans_linear_workspace_bytes(0, 100, 64, 32, 1)
    need_g = lib.kmeans_linear_workspace_bytes(1, 100, 64, 32, 1)
    assert need > 0 and need_g >= need + 100 * 64 * 2
    for sizes in ((2, 1, 1, 1, 1), (0, -1, 1, 1, 1), (0, 1, 0, 1, 1), (0, 1, 1, 0, 1), (0, 1, 1, 1, 1025),
                  (0, 1, 2 ** 30, 1, 4)):
        assert lib.kmeans_linear_workspace_bytes(*sizes) == 0
    lin = lambda x=F, ldx=32, w=F, b=None, res=None, ldr=0, dt=2, act=0, off=None, m=100, n=64, k=32, E=1, y=F, \
        pre=None, ws=W, wsb=1 << 40: lib.kmeans_linear(x, ldx, w, b, res, ldr, dt, act, off, m, n, k, E, y, pre, ws,
                                                       wsb, None)
    assert lin(x=None) == BAD and lin(w=None) == BAD and lin(y=None) == BAD and lin(ldx=31) == BAD
    assert lin(act=5) == BAD and lin(act=-1) == BAD and lin(dt=7) == BAD and lin(res=F, ldr=63) == BAD
    assert lin(E=2) == BAD  # experts without offsets
    assert lin(off=odd, E=2) == BAD and lin(x=odd) == BAD and lin(pre=odd) == BAD
    assert lin(dt=0) == NO and lin(off=F, E=1025) == NO and lin(w=ctypes.c_void_p(0x10008)) == NO
    assert lin(wsb=need - 1) == km.KMEANS_ERR_WORKSPACE and lin(ws=None) == km.KMEANS_ERR_WORKSPACE
    grad = lambda dy=F, ld=64, x=F, ldx=32, w=F, pre=F, dt=1, act=4, off=None, m=100, n=64, k=32, E=1, dx=F, dw=F, \
        db=F, wsb=1 << 40: lib.kmeans_linear_grad(dy, ld, x, ldx, w, pre, dt, act, off, m, n, k, E, dx, dw, db, W, wsb,
                                                  None)
    assert grad(dy=None) == BAD and grad(ld=63) == BAD and grad(pre=None) == BAD and grad(x=None) == BAD
    assert grad(w=None) == BAD and grad(db=odd) == BAD and grad(dt=0) == NO
    assert grad(w=ctypes.c_void_p(0x10008)) == NO
    assert grad(wsb=need_g - 1) == km.KMEANS_ERR_WORKSPACE


def test_expert_binding_refuses_what_is_not_on_the_gpu(km):
    import torch
    x, ids = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int64)
    for call in (lambda: km.kmeans_route(ids, 4), lambda: km.kmeans_route_gather(x, ids.int(), ids.int()),
                 lambda: km.kmeans_route_combine(x, ids.int(), ids.int()),
                 lambda: km.kmeans_linear(x.half(), x.half())):
        with pytest.raises(ValueError, match="CUDA device"):
            call()
    with pytest.raises(TypeError, match="int32 or int64"):
        km.kmeans_route(x, 4)
    with pytest.raises(km.KMeansError):
        km.route_workspace(4, 33, 4, device="cpu")
    with pytest.raises(km.KMeansError):
        km.linear_workspace(km.OP_LINEAR, 4, 0, 8, device="cpu")

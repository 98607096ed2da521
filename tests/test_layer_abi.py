"""Host-side checks of the gate, layer norm and cross entropy entry points:
argument validation before anything touches the GPU, workspace sizes, and what
the binding refuses.  No kernel runs here (no GPU needed)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def km():
    from distance_argmin_gb300 import build as b
    b.build()
    import distance_argmin_gb300 as km
    km.load()
    return km


F = ctypes.c_void_p(0x10000)   # never dereferenced: validation fails first
W = ctypes.c_void_p(0x100000)  # 256-byte aligned
ODD = ctypes.c_void_p(0x10001)
TWO = ctypes.c_void_p(0x10002)
EIGHT = ctypes.c_void_p(0x10008)
NAN, INF = float("nan"), float("inf")


def test_the_gate_validates_on_the_host(km):
    lib = km.load()
    BAD, NO, OK = km.KMEANS_ERR_INVALID_ARG, km.KMEANS_ERR_UNSUPPORTED, km.KMEANS_OK
    assert km.GATE_MAX_GROUPS == 32

    def gate(l=F, ld=64, dt=2, kind=0, b=None, n=10, E=64, k=4, G=1, kg=1, scale=1.0, ids=F, w=F):
        return lib.kmeans_gate(l, ld, dt, kind, b, n, E, k, G, kg, 1, scale, ids, w, None)

    assert gate(l=None) == BAD and gate(ids=None) == BAD and gate(w=None) == BAD and gate(ld=63) == BAD
    assert gate(dt=3) == BAD and gate(kind=2) == BAD and gate(kind=-1) == BAD and gate(l=ODD) == BAD
    assert gate(l=TWO, dt=0) == BAD and gate(b=TWO) == BAD and gate(ids=TWO) == BAD and gate(w=TWO) == BAD
    assert gate(n=-1) == BAD and gate(n=2 ** 31) == BAD and gate(E=0) == BAD and gate(k=65) == BAD and gate(k=-1) == BAD
    assert gate(G=0) == BAD and gate(G=3) == BAD and gate(G=4, kg=5) == BAD and gate(G=4, kg=0) == BAD
    assert gate(scale=NAN) == BAD and gate(scale=INF) == BAD
    assert gate(ld=5000, E=4097) == NO and gate(k=33) == NO and gate(G=64) == NO
    assert gate(n=0, l=None, ids=None, w=None) == OK and gate(k=0, ids=None, w=None) == OK  # nothing enqueued

    def grad(d=F, l=F, ld=64, dt=1, kind=1, ids=F, n=10, E=64, k=4, scale=1.0, out=F):
        return lib.kmeans_gate_grad(d, l, ld, dt, kind, ids, n, E, k, 0, scale, out, None)

    assert grad(d=None) == BAD and grad(l=None) == BAD and grad(ids=None) == BAD and grad(out=None) == BAD
    assert grad(ld=63) == BAD and grad(out=ODD) == BAD and grad(d=TWO) == BAD and grad(k=65) == BAD and grad(dt=9) == BAD
    assert grad(k=33) == NO and grad(ld=5000, E=4097) == NO
    assert grad(n=0, d=None, l=None, ids=None, out=None) == OK


def test_the_layer_norm_validates_on_the_host(km):
    lib = km.load()
    BAD, NO, OK, WS = km.KMEANS_ERR_INVALID_ARG, km.KMEANS_ERR_UNSUPPORTED, km.KMEANS_OK, km.KMEANS_ERR_WORKSPACE

    def norm(x=F, ld=32, dt=2, w=None, b=None, eps=1e-5, n=10, d=32, y=F, mean=None, rstd=None):
        return lib.kmeans_layernorm(x, ld, dt, w, b, eps, n, d, y, mean, rstd, None)

    assert norm(x=None) == BAD and norm(y=None) == BAD and norm(ld=31) == BAD and norm(dt=3) == BAD
    assert norm(x=ODD) == BAD and norm(w=ODD) == BAD and norm(b=ODD) == BAD and norm(mean=TWO) == BAD
    assert norm(rstd=TWO) == BAD and norm(x=TWO, dt=0) == BAD and norm(d=0) == BAD and norm(n=-1) == BAD
    assert norm(eps=-1e-9) == BAD and norm(eps=NAN) == BAD and norm(eps=INF) == BAD
    assert norm(d=km.ROUTE_MAX_WIDTH + 1, ld=2 ** 30) == NO
    assert norm(n=0, x=None, y=None) == OK
    need = lib.kmeans_layernorm_workspace_bytes(10, 32)
    assert need > 0 and lib.kmeans_layernorm_workspace_bytes(0, 1) > 0
    # the sums do not grow with the rows
    assert lib.kmeans_layernorm_workspace_bytes(2 ** 31 - 1, 4096) < 2 ** 26
    for sizes in ((-1, 4), (4, 0), (2 ** 31, 4), (4, km.ROUTE_MAX_WIDTH + 1)):
        assert lib.kmeans_layernorm_workspace_bytes(*sizes) == 0

    def grad(dy=F, ldy=32, x=F, ldx=32, dt=1, mean=F, rstd=F, w=None, res=None, ldr=0, n=10, d=32, dx=F, dw=F, db=F,
             ws=W, wsb=1 << 40):
        return lib.kmeans_layernorm_grad(dy, ldy, x, ldx, dt, mean, rstd, w, res, ldr, n, d, dx, dw, db, ws, wsb, None)

    assert grad(dy=None) == BAD and grad(x=None) == BAD and grad(mean=None) == BAD and grad(rstd=None) == BAD
    assert grad(ldy=31) == BAD and grad(ldx=31) == BAD and grad(res=F, ldr=31) == BAD and grad(dx=ODD) == BAD
    assert grad(dw=ODD) == BAD and grad(db=ODD) == BAD and grad(mean=TWO) == BAD and grad(dt=-1) == BAD
    assert grad(d=km.ROUTE_MAX_WIDTH + 1, ldy=2 ** 30, ldx=2 ** 30) == NO
    assert grad(wsb=need - 1) == WS and grad(ws=None) == WS and grad(ws=ODD) == WS


def test_the_cross_entropy_validates_on_the_host(km):
    lib = km.load()
    BAD, NO, WS = km.KMEANS_ERR_INVALID_ARG, km.KMEANS_ERR_UNSUPPORTED, km.KMEANS_ERR_WORKSPACE
    assert km.CROSS_ENTROPY_MAX_WIDTH == 32768
    size = lib.kmeans_cross_entropy_workspace_bytes
    need, need_g = size(0, 100, 1000, 64), size(1, 100, 1000, 64)
    assert 0 < need <= need_g and size(0, 0, 1, 1) > 0
    for sizes in ((2, 1, 1, 1), (0, -1, 1, 1), (0, 1, 0, 1), (0, 1, 1, 0), (0, 1, 1, 32769), (0, 2 ** 22, 2 ** 21, 8)):
        assert size(*sizes) == 0
    # no m * n logits: an eighth of a byte per logit forward, half a gigabyte of dz at most
    assert size(0, 8192, 131072, 64) < 8192 * 131072 / 6
    assert size(1, 8192, 131072, 64) < 2 ** 30

    def xent(x=F, ld=64, w=F, dt=2, labels=F, b=8, scale=1.0, m=100, n=1000, k=64, loss=F, lse=F, ws=W, wsb=1 << 50):
        return lib.kmeans_cross_entropy(x, ld, w, dt, labels, b, scale, m, n, k, loss, lse, ws, wsb, None)

    assert xent(x=None) == BAD and xent(w=None) == BAD and xent(labels=None) == BAD and xent(loss=None) == BAD
    assert xent(lse=None) == BAD and xent(ld=63) == BAD and xent(dt=5) == BAD and xent(b=2) == BAD
    assert xent(x=ODD) == BAD and xent(w=ODD) == BAD and xent(loss=TWO) == BAD and xent(lse=TWO) == BAD
    assert xent(labels=ctypes.c_void_p(0x10004)) == BAD and xent(b=4, labels=TWO) == BAD
    assert xent(scale=0.0) == BAD and xent(scale=-1.0) == BAD and xent(scale=NAN) == BAD and xent(scale=INF) == BAD
    assert xent(m=-1) == BAD and xent(n=0) == BAD and xent(k=0) == BAD and xent(m=2 ** 22, n=2 ** 21, k=8, ld=8) == BAD
    assert xent(dt=0) == NO and xent(k=32769, ld=40000) == NO and xent(w=EIGHT) == NO
    assert xent(wsb=need - 1) == WS and xent(ws=None) == WS and xent(ws=ODD) == WS

    def grad(d=F, x=F, ld=64, w=F, dt=1, labels=F, b=4, lse=F, scale=1.0, m=100, n=1000, k=64, dx=F, dw=F, wsb=1 << 50):
        return lib.kmeans_cross_entropy_grad(d, x, ld, w, dt, labels, b, lse, scale, m, n, k, dx, dw, W, wsb, None)

    assert grad(d=None) == BAD and grad(lse=None) == BAD and grad(x=None) == BAD and grad(w=None) == BAD
    assert grad(dx=ODD) == BAD and grad(dw=ODD) == BAD and grad(d=TWO) == BAD and grad(b=3) == BAD
    assert grad(dt=0) == NO and grad(w=EIGHT) == NO and grad(wsb=need_g - 1) == WS


@pytest.mark.parametrize("scale", [1.75 * 2.0 ** 127, 3e38])
def test_a_scale_whose_product_with_the_logits_unit_overflows_is_refused(km, scale):
    lib, BAD = km.load(), km.KMEANS_ERR_INVALID_ARG
    # finite, but times 1 / ln 2 it is not: a row of zeros would lose log(n) to NaN
    a = [F, 64, F, 2, F, 8]
    assert lib.kmeans_cross_entropy(*a, scale, 100, 1000, 64, F, F, W, 1 << 50, None) == BAD
    assert lib.kmeans_cross_entropy_grad(F, *a, F, scale, 100, 1000, 64, F, F, W, 1 << 50, None) == BAD


def test_the_binding_refuses_what_is_not_on_the_gpu(km):
    import torch
    x, i = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32)
    v = torch.zeros(4)
    for call in (lambda: km.kmeans_gate(x, 2), lambda: km.kmeans_gate_grad(x[:, :2], x, i),
                 lambda: km.kmeans_layernorm(x), lambda: km.kmeans_layernorm_grad(x, x, v, v),
                 lambda: km.kmeans_cross_entropy(x.half(), x.half(), i[:, 0]),
                 lambda: km.kmeans_cross_entropy_grad(v, x.half(), x.half(), i[:, 0], v)):
        with pytest.raises(ValueError, match="CUDA device"):
            call()
    for call in (lambda: km.layernorm_workspace(4, 0, device="cpu"),
                 lambda: km.cross_entropy_workspace(km.OP_CROSS_ENTROPY, 4, 0, 8, device="cpu")):
        with pytest.raises(km.KMeansError):
            call()


@pytest.mark.parametrize("n,k", [(1, 1), (1000, 64), (131072, 515)])
def test_a_batch_of_no_rows_has_workspaces_and_a_gradient(km, n, k):
    lib = km.load()
    need, need_g = (lib.kmeans_cross_entropy_workspace_bytes(g, 0, n, k) for g in (0, 1))
    assert 0 < need <= need_g
    # the sizes are worked out before the workspace is refused, and nothing is enqueued
    a = [None, k, None, 2, None, 8]
    for wsb in (0, need_g - 1):
        assert lib.kmeans_cross_entropy_grad(None, *a, None, 1.0, 0, n, k, F, F, W, wsb, None) == km.KMEANS_ERR_WORKSPACE


@pytest.mark.parametrize("m", [1, 64, 65, 128, 1000, 8192, 2 ** 17, 2 ** 20])
@pytest.mark.parametrize("n", [1, 257, 4096, 10007, 131072])
@pytest.mark.parametrize("k", [64, 513, 4096])
def test_the_cross_entropy_workspace_keeps_to_what_the_header_says(km, m, n, k):
    lib = km.load()
    forward, both = (lib.kmeans_cross_entropy_workspace_bytes(g, m, n, k) for g in (0, 1))
    rows, wide = (m + 31) // 32 * 32, (k + 7) // 8 * 8
    # 16 bytes a row and 4 for its label's logit, x once (and w, where it has to be brought to 16 bytes), 8 bytes per 16
    # classes (a last unit of 64 has four parts, however few its classes); 16 KiB of status words and of space between
    kept = 24 * m + 2 * m * wide + (2 * n * wide if k % 8 else 0) + (1 << 14)
    assert 0 < forward <= kept + rows * (n / 16 + 4) * 8
    # a piece is at most 8 classes more than n, 2^28 values or 2048 classes; dx's sums: a split product has at most 76
    # units of 256 x 256, or 76 parts of one unit; dw's: one of m / 32768 chunks of a piece
    piece = min(n + 8, 32768, max(2048, 2 ** 28 // m + 256))
    sums = 4 * max(m, 256 * 76) * max(k, 256)
    chunks = 4 * ((m + 32767) // 32768 if m > 32768 else 0) * piece * k
    assert forward <= both <= max(kept + rows * (n / 16 + 4) * 8, kept + 2 * m * wide + 2 * m * piece + sums + chunks)

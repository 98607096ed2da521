"""The experts' matrix products on the GPU against a plain implementation in
float64.

Bounds, fixed before any run.  A sum of K products: the tensor cores add 16 of
them at a time into a float32 accumulator, cutting off what does not fit, so
each of the K / 16 additions costs up to 2^-23 of the sum of the products'
magnitudes S, and the 16 products inside one are aligned to the largest with
as much again: (K / 16 + 16) 2^-23 S (plain float32 additions cost less).  The
activations and their slopes change by at most 1.2 times their argument's
change and are within 2^-19 (|z| + 1) of their formula in float32.  A result
kept in b significant bits is within 2^-b of itself (float16 also within
2^-25).  The gradient's products take dz in b bits: 2^-b |dz| (and 2^-25 in
float16) per factor.
"""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

BITS = {torch.float16: 11, torch.bfloat16: 8}
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 0.0}
DTYPES = [torch.float16, torch.bfloat16]
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


def act(z, name):
    if name == "relu":
        return z.clamp(min=0)
    if name == "gelu":
        return z * 0.5 * torch.special.erfc(-z / math.sqrt(2))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if name == "silu":
        return z * torch.sigmoid(z)
    return z


def normal(shape, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def within(got, want, size, steps, dtype, extra=0.0):
    bound = steps * 2.0 ** -23 * size + extra
    bound = bound + 2.0 ** -BITS[dtype] * (want.abs() + bound) + TINY[dtype]
    off = (got.double() - want).abs()
    assert bool((off <= bound).all()), f"off by {(off - bound).max().item():.3e} more than the bound"


def steps_for(k):
    return k / 16 + 17


def group_counts(m, n_experts, dropped, seed):
    """Rows per expert with empty experts among them."""
    r = np.random.RandomState(seed)
    share = np.where(r.rand(n_experts) < 0.3, 0.0, r.rand(n_experts) ** 2)
    if share.sum() == 0:
        share[-1] = 1.0
    return r.multinomial(m - dropped, share / share.sum())


def as_offsets(counts):
    return torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).cuda()


def plain(x, w, bias, residual, edges, name):
    m, n = x.shape[0], w.shape[1]
    z = torch.zeros(m, n, dtype=torch.float64, device="cuda")
    size, y = torch.zeros_like(z), torch.zeros_like(z)
    for e in range(w.shape[0]):
        a, b = edges[e], edges[e + 1]
        z[a:b] = x[a:b].double() @ w[e].double().t()
        size[a:b] = x[a:b].double().abs() @ w[e].double().abs().t()
        if bias is not None:
            z[a:b] += bias[e].double()
            size[a:b] += bias[e].double().abs()
        y[a:b] = act(z[a:b], name)
        if residual is not None:
            y[a:b] += residual[a:b].double()
    return z, y, size


def check_forward(km, x, w, bias, residual, offsets, name, pre):
    ws = km.linear_workspace(km.OP_LINEAR, x.shape[0], w.shape[-2], w.shape[-1], w.shape[0] if w.dim() == 3 else 1)
    y, z = km.kmeans_linear(x, w, bias=bias, residual=residual, offsets=offsets, activation=name, save_pre=pre, ws=ws)
    assert km.kmeans_device_status(ws) == km.KMEANS_OK
    w3 = w if w.dim() == 3 else w[None]
    b2 = bias if bias is None or bias.dim() == 2 else bias[None]
    edges = [0, x.shape[0]] if offsets is None else offsets.tolist()
    want_z, want_y, size = plain(x, w3, b2, residual, edges, name)
    steps = steps_for(x.shape[1])
    last = edges[-1]
    if pre:
        within(z, want_z, size, steps, x.dtype)
    else:
        assert z is None
    extra = 2.0 ** -19 * (want_z.abs() + 1)
    extra[last:] = 0
    if residual is not None:
        extra = extra + 2.0 ** -23 * residual.double().abs()
    within(y, want_y, 1.2 * size, steps, x.dtype, extra)
    assert not y[last:].any()
    return y


DENSE = [(1, 8, 8), (1, 64, 512), (3, 33, 17), (8, 128, 64), (17, 1000, 520), (40, 264, 1032), (129, 257, 72),
         (300, 515, 333), (512, 512, 2048), (257, 96, 4104), (1000, 136, 8)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,n,k", DENSE)
def test_dense_forward(gpu_lib, m, n, k, dtype):
    x, w = normal((m, k), dtype, 1), normal((n, k), dtype, 2, k ** -0.5)
    bias, res = normal((n,), dtype, 3), normal((m, n), dtype, 4)
    name = ACTS[(m + n) % 5]
    check_forward(gpu_lib, x, w, bias, res, None, name, True)
    check_forward(gpu_lib, x, w, None, None, None, "none", False)


@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("m", [5, 200])
def test_every_activation_over_its_whole_range(gpu_lib, m, name):
    x, w = normal((m, 64), torch.float16, 5), normal((80, 64), torch.float16, 6, 1.0)
    x[::3] *= 0.01
    check_forward(gpu_lib, x, w, normal((80,), torch.float16, 7), normal((m, 80), torch.float16, 8), None, name, True)


GROUPS = [(1, 4, 0, 64, 64), (7, 16, 1, 48, 72), (24, 64, 0, 200, 512), (100, 3, 100, 64, 64), (130, 1, 5, 72, 40),
          (513, 9, 13, 264, 136), (700, 40, 0, 33, 51), (2000, 6, 100, 320, 1032), (1500, 300, 1, 24, 16)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,n_experts,dropped,n,k", GROUPS)
def test_grouped_forward(gpu_lib, m, n_experts, dropped, n, k, dtype):
    counts = group_counts(m, n_experts, dropped, m + n)
    x, w = normal((m, k), dtype, 1), normal((n_experts, n, k), dtype, 2, k ** -0.5)
    bias, res = normal((n_experts, n), dtype, 3), normal((m, n), dtype, 4)
    offsets = as_offsets(counts)
    last = m - dropped
    x[last:] = float("nan")  # rows of no expert hold anything
    res[last:] = float("inf")
    clean = res.clone()
    clean[last:] = 0
    y, _ = gpu_lib.kmeans_linear(x, w, bias=bias, residual=res, offsets=offsets, activation="silu")
    x[last:] = 0
    ref = check_forward(gpu_lib, x, w, bias, clean, offsets, "silu", True)
    assert torch.equal(y, ref)


@pytest.mark.parametrize("m,n_experts,n,k", [(20, 4, 64, 64), (600, 4, 64, 136), (600, 4, 72, 35)])
def test_infinities_stay_in_their_row_and_their_expert(gpu_lib, m, n_experts, n, k):
    counts = np.full(n_experts, m // n_experts)
    offsets = as_offsets(counts)
    edges = offsets.tolist()
    x, w = normal((m, k), torch.bfloat16, 1), normal((n_experts, n, k), torch.bfloat16, 2, k ** -0.5)
    dy = normal((m, n), torch.bfloat16, 3)
    y0, _ = gpu_lib.kmeans_linear(x, w, offsets=offsets)
    dx0, dw0, db0 = gpu_lib.kmeans_linear_grad(dy, x, w, offsets=offsets)
    x1, w1, dy1 = x.clone(), w.clone(), dy.clone()
    bad_row = edges[1]           # the first row of expert 1, next to expert 0's last
    x1[bad_row, 0] = float("inf")
    x1[edges[3] - 1, 1] = float("nan")
    w1[3, 0, 0] = float("nan")   # next to expert 2's last feature
    dy1[bad_row, 0] = float("nan")
    y1, _ = gpu_lib.kmeans_linear(x1, w1, offsets=offsets)
    dx1, dw1, db1 = gpu_lib.kmeans_linear_grad(dy1, x1, w1, offsets=offsets)
    rows = torch.ones(m, dtype=torch.bool)
    rows[[bad_row, edges[3] - 1]] = False
    rows[edges[3]:] = False
    assert torch.equal(y1[rows.cuda()], y0[rows.cuda()]) and torch.equal(dx1[rows.cuda()], dx0[rows.cuda()])
    assert not torch.isfinite(y1[bad_row]).all() and torch.isnan(dx1[bad_row]).all()
    assert torch.equal(y1[edges[3]:, 1:], y0[edges[3]:, 1:]) and torch.isnan(y1[edges[3]:, 0]).all()
    assert torch.equal(dw1[0], dw0[0]) and torch.equal(db1[[0, 2, 3]], db0[[0, 2, 3]])
    assert torch.equal(dw1[3], dw0[3]) and torch.isnan(dw1[1, 0]).all() and torch.isnan(db1[1, 0])


def test_offsets_that_run_backwards_or_past_the_rows_are_cut(gpu_lib):
    m, n, k = 90, 40, 24
    x, w = normal((m, k), torch.bfloat16, 1), normal((4, n, k), torch.bfloat16, 2)
    dy = normal((m, n), torch.bfloat16, 3)
    bad = torch.tensor([0, 50, 20, 2 ** 30, 60], dtype=torch.int32, device="cuda")
    cut = torch.tensor([0, 50, 50, 90, 90], dtype=torch.int32, device="cuda")
    for a, b in zip(gpu_lib.kmeans_linear(x, w, offsets=bad, save_pre=True),
                    gpu_lib.kmeans_linear(x, w, offsets=cut, save_pre=True)):
        assert torch.equal(a, b)
    for a, b in zip(gpu_lib.kmeans_linear_grad(dy, x, w, offsets=bad), gpu_lib.kmeans_linear_grad(dy, x, w, offsets=cut)):
        assert torch.equal(a, b)


def check_gradient(km, dy, x, w, pre, offsets, name):
    w3 = w if w.dim() == 3 else w[None]
    m, n, k, n_experts = x.shape[0], w3.shape[1], w3.shape[2], w3.shape[0]
    ws = km.linear_workspace(km.OP_LINEAR_GRAD, m, n, k, n_experts)
    got = km.kmeans_linear_grad(dy, x, w, pre=pre, offsets=offsets, activation=name, ws=ws)
    assert km.kmeans_device_status(ws) == km.KMEANS_OK
    dx, dw, db = got[0], got[1].view(w3.shape), got[2].view(n_experts, n)
    edges = [0, m] if offsets is None else offsets.tolist()
    z = pre.double().requires_grad_() if pre is not None else torch.zeros(m, n, dtype=torch.float64, device="cuda")
    if name == "none":
        sl = torch.ones_like(z)
    else:
        sl, = torch.autograd.grad(act(z, name).sum(), z)
        z = z.detach()
    if name == "relu":
        sl = (pre > 0).double()  # 0 at 0
    g = dy.double()
    dz = g * sl
    slope_err = g.abs() * 2.0 ** -19 * (z.abs() + 1) if name not in ("none", "relu") else torch.zeros_like(dz)
    kept = slope_err + (2.0 ** -BITS[dy.dtype] * dz.abs() + TINY[dy.dtype] if name not in ("none", "relu") else 0)
    wd, xd = w3.double(), x.double()
    for e in range(n_experts):
        a, b = edges[e], edges[e + 1]
        within(dx[a:b], dz[a:b] @ wd[e], dz[a:b].abs() @ wd[e].abs(), steps_for(n), dy.dtype,
               kept[a:b] @ wd[e].abs())
        within(dw[e], dz[a:b].t() @ xd[a:b], dz[a:b].abs().t() @ xd[a:b].abs(), steps_for(b - a), dy.dtype,
               kept[a:b].t() @ xd[a:b].abs())
        within(db[e], dz[a:b].sum(0), dz[a:b].abs().sum(0), steps_for(b - a), dy.dtype, slope_err[a:b].sum(0))
        if a == b:
            assert not dw[e].any() and not db[e].any()
    assert not dx[edges[-1]:].any()
    return got


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,n,k", DENSE)
def test_dense_gradient(gpu_lib, m, n, k, dtype):
    x, w = normal((m, k), dtype, 1), normal((n, k), dtype, 2, k ** -0.5)
    dy, pre = normal((m, n), dtype, 3), normal((m, n), dtype, 4, 2.0)
    check_gradient(gpu_lib, dy, x, w, pre, None, ACTS[(m + n) % 5])
    check_gradient(gpu_lib, dy, x, w, None, None, "none")


@pytest.mark.parametrize("name", ACTS)
def test_every_slope_over_its_whole_range(gpu_lib, name):
    pre = normal((200, 80), torch.float16, 4, 4.0)
    pre[0] = 0
    pre[1] = -0.0
    check_gradient(gpu_lib, normal((200, 80), torch.float16, 3), normal((200, 64), torch.float16, 1),
                   normal((80, 64), torch.float16, 2), pre, None, name)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,n_experts,dropped,n,k", GROUPS)
def test_grouped_gradient(gpu_lib, m, n_experts, dropped, n, k, dtype):
    counts = group_counts(m, n_experts, dropped, m + n)
    x, w = normal((m, k), dtype, 1), normal((n_experts, n, k), dtype, 2, k ** -0.5)
    dy, pre = normal((m, n), dtype, 3), normal((m, n), dtype, 4)
    last = m - dropped
    offsets = as_offsets(counts)
    for t in (x, dy, pre):
        t[last:] = float("nan")
    got = gpu_lib.kmeans_linear_grad(dy, x, w, pre=pre, offsets=offsets, activation="gelu")
    for t in (x, dy, pre):
        t[last:] = 0
    ref = check_gradient(gpu_lib, dy, x, w, pre, offsets, "gelu")
    for a, b in zip(got, ref):
        assert torch.equal(a, b)


def test_only_what_is_asked_for(gpu_lib):
    x, w, dy = (normal(s, torch.bfloat16, i) for i, s in enumerate([(70, 40), (24, 40), (70, 24)]))
    full = gpu_lib.kmeans_linear_grad(dy, x, w)
    for keep in range(3):
        got = gpu_lib.kmeans_linear_grad(dy, x, w, need_dx=keep == 0, need_dw=keep == 1, need_db=keep == 2)
        assert [g is not None for g in got] == [keep == i for i in range(3)]
        assert torch.equal(got[keep], full[keep])


def test_gradient_agrees_with_differences(gpu_lib):
    """Differences of the float64 formula, whose gradient the kernels give in
    16 bits: central differences over h are off by h^2 / 6 times the third
    derivative (below 2 here), and the kernels by 2^-7 of the terms."""
    m, n, k, h = 12, 16, 8, 1e-3
    x, w = normal((m, k), torch.bfloat16, 1), normal((n, k), torch.bfloat16, 2)
    dy = normal((m, n), torch.bfloat16, 3)
    _, pre = gpu_lib.kmeans_linear(x, w, activation="gelu_tanh", save_pre=True)
    dx, dw, db = gpu_lib.kmeans_linear_grad(dy, x, w, pre=pre, activation="gelu_tanh")

    def loss(x, w, b):
        return (act(x @ w.t() + b, "gelu_tanh") * dy.double()).sum().item()

    args = [x.double(), w.double(), torch.zeros(n, dtype=torch.float64, device="cuda")]
    size = dy.double().abs().sum().item() / 4
    r = np.random.RandomState(1)
    for which, grad in enumerate((dx, dw, db)):
        for _ in range(8):
            at = tuple(r.randint(s) for s in grad.shape)
            up, down = [a.clone() for a in args], [a.clone() for a in args]
            up[which][at] += h
            down[which][at] -= h
            diff = (loss(*up) - loss(*down)) / (2 * h)
            assert abs(diff - grad[at].item()) <= 2.0 ** -6 * (abs(diff) + size / n) + 1e-4


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m", [6, 150])
def test_strided_and_unaligned_inputs(gpu_lib, m, dtype):
    n, k = 72, 64
    w = normal((n, k), dtype, 2)
    for pitch, first in ((80, 8), (71, 3)):
        x = normal((m, pitch), dtype, 1)[:, first:first + k]
        res = normal((m, n + pitch), dtype, 4)[:, first:first + n]
        dy = normal((m, n + pitch), dtype, 5)[:, first:first + n]
        a, _ = gpu_lib.kmeans_linear(x, w, residual=res, activation="relu")
        b, _ = gpu_lib.kmeans_linear(x.contiguous(), w, residual=res.contiguous(), activation="relu")
        assert torch.equal(a, b)
        for a, b in zip(gpu_lib.kmeans_linear_grad(dy, x, w), gpu_lib.kmeans_linear_grad(dy.contiguous(),
                                                                                          x.contiguous(), w)):
            assert torch.equal(a, b)
    flat = torch.empty(n * k + 1, dtype=dtype, device="cuda")
    off = flat[1:].view(n, k)
    off.copy_(w)
    x = normal((m, k), dtype, 1)
    ref, _ = gpu_lib.kmeans_linear(x, w)
    for call in (lambda: gpu_lib.kmeans_linear(x, off), lambda: gpu_lib.kmeans_linear_grad(ref, x, off)):
        with pytest.raises(gpu_lib.KMeansError) as err:  # w has to start on 16 bytes
            call()
        assert err.value.status == gpu_lib.KMEANS_ERR_UNSUPPORTED
    out = torch.empty(m * n + 1, dtype=dtype, device="cuda")[1:].view(m, n)
    assert torch.equal(gpu_lib.kmeans_linear(x, w, y=out)[0], ref)


def test_same_bits_from_call_to_call_and_on_another_stream(gpu_lib):
    m, n, k = 333, 264, 520
    offsets = as_offsets(group_counts(m, 5, 3, 0))
    x, w, dy = normal((m, k), torch.bfloat16, 1), normal((5, n, k), torch.bfloat16, 2), normal((m, n), torch.bfloat16, 3)
    pre = normal((m, n), torch.bfloat16, 4)

    def both(stream=None):
        y, _ = gpu_lib.kmeans_linear(x, w, offsets=offsets, activation="gelu", stream=stream)
        return (y, *gpu_lib.kmeans_linear_grad(dy, x, w, pre=pre, offsets=offsets, activation="gelu", stream=stream))

    ref = both()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (None, side):
        got = both(stream)
        torch.cuda.synchronize()
        for a, b in zip(got, ref):
            assert torch.equal(a, b)


def test_forward_and_gradient_replay_in_a_graph(gpu_lib):
    m, n, k = 100, 64, 128
    x, w, dy = normal((m, k), torch.float16, 1), normal((n, k), torch.float16, 2), normal((m, n), torch.float16, 3)
    wf, wg = gpu_lib.linear_workspace(gpu_lib.OP_LINEAR, m, n, k), gpu_lib.linear_workspace(gpu_lib.OP_LINEAR_GRAD, m, n, k)
    y, pre = gpu_lib.kmeans_linear(x, w, activation="silu", save_pre=True, ws=wf)
    dx, dw, db = gpu_lib.kmeans_linear_grad(dy, x, w, pre=pre, activation="silu", ws=wg)
    ref = [t.clone() for t in (y, pre, dx, dw, db)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gpu_lib.kmeans_linear(x, w, activation="silu", y=y, pre=pre, ws=wf)
        gpu_lib.kmeans_linear_grad(dy, x, w, pre=pre, activation="silu", dx=dx, dw=dw, db=db, ws=wg)
    for t in (y, pre, dx, dw, db):
        t.zero_()
    g.replay()
    torch.cuda.synchronize()
    for a, b in zip((y, pre, dx, dw, db), ref):
        assert torch.equal(a, b)


def test_no_rows(gpu_lib):
    x, w = torch.empty(0, 16, dtype=torch.bfloat16, device="cuda"), normal((3, 24, 16), torch.bfloat16, 1)
    offsets = torch.zeros(4, dtype=torch.int32, device="cuda")
    y, pre = gpu_lib.kmeans_linear(x, w, offsets=offsets, save_pre=True)
    assert y.shape == (0, 24) and pre.shape == (0, 24)
    dw = torch.full_like(w, 3.0)
    db = torch.full((3, 24), 3.0, dtype=torch.bfloat16, device="cuda")
    dx, dw, db = gpu_lib.kmeans_linear_grad(y, x, w, offsets=offsets, dw=dw, db=db)
    assert dx.shape == (0, 16) and not dw.any() and not db.any()


@pytest.mark.parametrize("rows", [3, 200])
def test_weights_of_more_than_two_to_the_31_values(gpu_lib, rows):
    n_experts, n, k = 35, 8192, 8192
    assert n_experts * n * k > 2 ** 31
    w = torch.zeros(n_experts, n, k, dtype=torch.bfloat16, device="cuda")
    w[-1] = normal((n, k), torch.bfloat16, 1, k ** -0.5)
    x = normal((rows, k), torch.bfloat16, 2)
    offsets = torch.zeros(n_experts + 1, dtype=torch.int32, device="cuda")
    offsets[-1] = rows
    y, _ = gpu_lib.kmeans_linear(x, w, offsets=offsets)
    ref, _ = gpu_lib.kmeans_linear(x, w[-1])
    assert torch.equal(y, ref) if rows > 100 else torch.allclose(y.float(), ref.float(), atol=0.05)
    dy = normal((rows, n), torch.bfloat16, 3)
    dx, dw, _ = gpu_lib.kmeans_linear_grad(dy, x, w, offsets=offsets, need_db=False)
    rdx, rdw, _ = gpu_lib.kmeans_linear_grad(dy, x, w[-1].contiguous(), need_db=False)
    within(dx, rdx.double(), rdx.double().abs(), 0, torch.bfloat16, 2.0 ** -8 * rdx.double().abs() + 1e-3)
    within(dw[-1], rdw.double(), rdw.double().abs(), 0, torch.bfloat16, 2.0 ** -8 * rdw.double().abs() + 1e-3)
    assert not dw[:-1].any()


def test_a_starved_pipeline_reports_a_timeout_and_the_next_call_works(gpu_lib, monkeypatch):
    x, w, dy = (normal(s, torch.bfloat16, i) for i, s in enumerate([(300, 128), (264, 128), (300, 264)]))
    wf = gpu_lib.linear_workspace(gpu_lib.OP_LINEAR, 300, 264, 128)
    wg = gpu_lib.linear_workspace(gpu_lib.OP_LINEAR_GRAD, 300, 264, 128)
    ref = (gpu_lib.kmeans_linear(x, w)[0], *gpu_lib.kmeans_linear_grad(dy, x, w))
    monkeypatch.setenv("KMEANS_GB300_TEST_STARVE_PIPELINE", "1")
    gpu_lib.kmeans_linear(x, w, ws=wf)
    assert gpu_lib.kmeans_device_status(wf) == gpu_lib.KMEANS_ERR_DEVICE_TIMEOUT
    gpu_lib.kmeans_linear_grad(dy, x, w, ws=wg)
    assert gpu_lib.kmeans_device_status(wg) == gpu_lib.KMEANS_ERR_DEVICE_TIMEOUT
    monkeypatch.delenv("KMEANS_GB300_TEST_STARVE_PIPELINE")
    got = (gpu_lib.kmeans_linear(x, w, ws=wf)[0], *gpu_lib.kmeans_linear_grad(dy, x, w, ws=wg))
    assert gpu_lib.kmeans_device_status(wf) == gpu_lib.KMEANS_OK == gpu_lib.kmeans_device_status(wg)
    for a, b in zip(got, ref):
        assert torch.equal(a, b)


@pytest.mark.parametrize("m,n,k", [(9_000_000, 16, 8), (200_000, 72, 40), (20_000, 512, 520), (3000, 33, 17)])
def test_the_weight_gradient_of_many_rows_keeps_its_bits(gpu_lib, m, n, k):
    """Sums over many rows: the accumulator's cut-off (up to 2^-23 of the running
    sum in each of its additions, 16 rows at a time) may not add up over all of
    them.  At most 32768 rows share an accumulator, so 2048 additions lose up to
    2^-12 of the largest running sum, which is the sum itself where it grows and
    within six standard deviations of the walk, the root of the sum of the
    products' squares, where it wanders; the result's rounding to 8 bits is up to
    2^-8 of it.  The forward pass of as many rows is checked beside it."""
    x, dy = normal((m, k), torch.bfloat16, 1), normal((m, n), torch.bfloat16, 2)
    x[:, 0] = x[:, 0].abs()  # sums that grow with the rows, next to ones that wander
    dy[:, 0] = dy[:, 0].abs()
    w = normal((n, k), torch.bfloat16, 3)
    ws = gpu_lib.linear_workspace(gpu_lib.OP_LINEAR_GRAD, m, n, k)
    dx, dw, db = gpu_lib.kmeans_linear_grad(dy, x, w, ws=ws)
    assert gpu_lib.kmeans_device_status(ws) == gpu_lib.KMEANS_OK
    def sums(f):
        return sum(f(dy[a:a + (1 << 20)].double(), x[a:a + (1 << 20)].double()) for a in range(0, m, 1 << 20))

    for got, exact, squares in ((dw, sums(lambda g, v: g.t() @ v), sums(lambda g, v: (g * g).t() @ (v * v))),
                                (db, sums(lambda g, v: g.sum(0)), sums(lambda g, v: (g * g).sum(0)))):
        bound = 2.0 ** -8 * exact.abs() + 2.0 ** -12 * (exact.abs() + 6 * squares.sqrt())
        assert bool(((got.double() - exact).abs() <= bound).all())
    last = slice(m - 500, m)
    within(dx[last], dy[last].double() @ w.double(), dy[last].double().abs() @ w.double().abs(), steps_for(n),
           torch.bfloat16)
    y, _ = gpu_lib.kmeans_linear(x, w)
    within(y[last], x[last].double() @ w.double().t(), x[last].double().abs() @ w.double().abs().t(), steps_for(k),
           torch.bfloat16)
    again = gpu_lib.kmeans_linear_grad(dy, x, w, need_dx=False, ws=ws)
    assert torch.equal(again[1], dw) and torch.equal(again[2], db)


def test_experts_of_one_and_of_several_chunks_of_rows(gpu_lib):
    # few output tiles: chunks are short here, so some experts take several
    counts = np.array([5000, 0, 300, 700, 1, 2600])
    m = int(counts.sum()) + 40
    x, dy = normal((m, 24), torch.float16, 1), normal((m, 40), torch.float16, 2)
    check_gradient(gpu_lib, dy, x, normal((6, 40, 24), torch.float16, 3), None, as_offsets(counts), "none")

"""Softmax cross entropy and its gradient on the GPU against float64.

Bounds, fixed before any run.  A logit is a sum of k products on the tensor
cores, within 6e-9 k + 2^-22 of the sum of its terms' magnitudes (cut off, not
rounded); ``dz`` below is the largest of a row.  The logarithm of the sum is
within dz + (2^-21 + |z| 2^-22) of its value, the loss within twice that.  In the
gradient a probability is within (that + 2^-21) of itself, dz is rounded to 16
bits (a relative 2^-b; float16 also 2^-38 of the largest dloss * scale, half its
smallest step 2^-24 after the power of two that takes that to 2^13), dW takes x
times a factor in [1/2, 1), rounded to 16 bits once more (2^-b of each term, and
2^-25, half float16's smallest step), the products cut off as the logits do, and
the result is rounded once.  The hardware's exp2 gives 0 for what is below 2^-126,
the smallest normal number: so much a probability may also be off by.
"""
import math

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

BITS = {torch.float16: 11, torch.bfloat16: 8}
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -126}
DTYPES = [torch.float16, torch.bfloat16]
CUT = 6e-9


def draw(m, n, k, dtype, seed, ignored=0.0, size=2.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    w = (torch.randn(n, k, generator=g, device="cuda") * size * k ** -0.5).to(dtype)
    labels = torch.randint(n, (m,), generator=g, device="cuda")
    x = (torch.randn(m, k, generator=g, device="cuda") + w[labels].float()).to(dtype)
    labels[torch.rand(m, generator=g, device="cuda") < ignored] = -1
    dloss = torch.rand(m, generator=g, device="cuda") / max(m, 1)
    return x, w, labels, dloss


def plain(x, w, labels, scale):
    """Logits, lse and loss of every row, and the logits' bound, in float64."""
    xd, wd = x.double(), w.double()
    z = scale * (xd @ wd.t())
    size = scale * (xd.abs() @ wd.abs().t())
    cut = ((CUT * x.shape[1] + 2.0 ** -22) * size).amax(1)
    lse = torch.logsumexp(z, 1)
    loss = lse - z.gather(1, labels.clamp(min=0)[:, None])[:, 0]
    return z, lse, loss, cut


def check_forward(km, x, w, labels, scale=1.0, **kw):
    loss, lse = km.kmeans_cross_entropy(x, w, labels, scale=scale, **kw)
    z, want_lse, want, cut = plain(x, w, labels, scale)
    live = (labels >= 0) & (labels < w.shape[0])
    assert loss.dtype == lse.dtype == torch.float32
    assert not loss[~live].any() and not lse[~live].any()
    off = cut + 2.0 ** -21 + z.abs().amax(1) * 2.0 ** -22
    assert bool(((lse.double() - want_lse).abs() <= off)[live].all())
    assert bool(((loss.double() - want).abs() <= 2 * off)[live].all())
    return loss, lse


def check_grad(km, dloss, x, w, labels, scale=1.0, **kw):
    _, lse = km.kmeans_cross_entropy(x, w, labels, scale=scale)
    dx, dw = km.kmeans_cross_entropy_grad(dloss, x, w, labels, lse, scale=scale, **kw)
    dt = x.dtype
    live = labels >= 0
    z, want_lse, _, cut = plain(x[live], w, labels[live], scale)
    g = scale * dloss[live].double()
    p = torch.exp(z - want_lse[:, None])
    hot = torch.nn.functional.one_hot(labels[live], w.shape[0]).double()
    dz = g[:, None] * (p - hot)
    rel = 2 * cut + 2.0 ** -20 + z.abs().amax(1) * 2.0 ** -21
    dz_off = g.abs()[:, None] * (p * rel[:, None] + 2.0 ** -126) + 2.0 ** -BITS[dt] * dz.abs() * (1 + rel[:, None])
    if dt is torch.float16 and g.numel():
        dz_off = dz_off + 2.0 ** -38 * g.abs().max()
    xd, wd = x[live].double(), w.double()
    want, off = torch.zeros(x.shape, dtype=torch.float64, device="cuda"), torch.zeros((), device="cuda")
    off = torch.zeros_like(want)
    want[live] = dz @ wd
    off[live] = dz_off @ wd.abs() + (CUT * w.shape[0] + 2.0 ** -20) * (dz.abs() @ wd.abs())
    bound = off + 1.01 * 2.0 ** -BITS[dt] * (want.abs() + off) + TINY[dt]
    assert bool(((dx.double() - want).abs() <= bound).all())
    want_w = dz.t() @ xd
    off_w = dz_off.t() @ xd.abs() + (CUT * x.shape[0] + 2.0 ** -20) * (dz.abs().t() @ xd.abs())
    # share * x: dz is then held as dz / share, which is at most twice as large
    off_w = off_w + 2.0 ** -BITS[dt] * ((dz.abs() + dz_off).t() @ xd.abs()) + 2 * TINY[dt] * dz.abs().sum(0)[:, None]
    bound = off_w + 1.01 * 2.0 ** -BITS[dt] * (want_w.abs() + off_w) + TINY[dt]
    assert bool(((dw.double() - want_w).abs() <= bound).all())
    return lse, dx, dw


SHAPES = [(1, 1, 1), (1, 2, 8), (1, 1000, 64), (2, 33, 17), (7, 256, 128), (24, 4096, 256), (64, 257, 520),
          (65, 31, 100), (257, 300, 72), (300, 10007, 130), (1031, 777, 515), (513, 5000, 64), (4097, 130, 40),
          (6000, 64, 16), (100, 40000, 24)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("ignored,scale", [(0.0, 1.0), (0.4, 0.3)])
def test_loss(gpu_lib, m, n, k, dtype, ignored, scale):
    x, w, labels, _ = draw(m, n, k, dtype, m + n, ignored)
    check_forward(gpu_lib, x, w, labels, scale)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("ignored,scale", [(0.0, 1.0), (0.4, 0.3)])
def test_gradient(gpu_lib, m, n, k, dtype, ignored, scale):
    x, w, labels, dloss = draw(m, n, k, dtype, m + n + 1, ignored)
    check_grad(gpu_lib, dloss, x, w, labels, scale)


@pytest.mark.parametrize("dtype", DTYPES)
def test_several_pieces_of_the_classes(gpu_lib, dtype):
    """66000 classes: three pieces, the last of another size; dx meets in float32."""
    x, w, labels, dloss = draw(70, 66003, 48, dtype, 5, 0.2)
    check_grad(gpu_lib, dloss, x, w, labels)


@pytest.mark.parametrize("m", [24, 70])
def test_a_large_class_matrix_off_16_bytes(gpu_lib, m):
    """34000 x 1001 values are brought to 16 bytes by a kernel of their own."""
    x, w, labels, dloss = draw(m, 34000, 1001, torch.bfloat16, 8, 0.1)
    check_forward(gpu_lib, x, w, labels)
    check_grad(gpu_lib, dloss, x, w, labels)


@pytest.mark.parametrize("dtype", DTYPES)
def test_more_rows_than_an_accumulator_takes(gpu_lib, dtype):
    x, w, labels, dloss = draw(70000, 40, 24, dtype, 6, 0.3)
    check_grad(gpu_lib, dloss, x, w, labels)
    labels[30000:] = -1  # the rows that count fill one chunk, though there was room for more
    check_grad(gpu_lib, dloss, x, w, labels)


@pytest.mark.parametrize("id_dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("m", [60, 5000])
def test_a_label_past_the_classes_is_ignored_and_reported(gpu_lib, id_dtype, m):
    x, w, labels, dloss = draw(m, 100, 32, torch.bfloat16, 3, 0.1)
    labels = labels.to(id_dtype)
    bad = labels.clone()
    bad[m // 2] = 100
    labels[m // 2] = -5
    ws = gpu_lib.cross_entropy_workspace(gpu_lib.OP_CROSS_ENTROPY_GRAD, m, 100, 32)
    want = gpu_lib.kmeans_cross_entropy(x, w, labels, ws=ws)
    assert gpu_lib.kmeans_device_status(ws) == gpu_lib.KMEANS_OK
    got = gpu_lib.kmeans_cross_entropy(x, w, bad, ws=ws)
    assert gpu_lib.kmeans_device_status(ws) == gpu_lib.KMEANS_ERR_DEVICE_LABEL
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    want = gpu_lib.kmeans_cross_entropy_grad(dloss, x, w, labels, got[1], ws=ws)
    assert gpu_lib.kmeans_device_status(ws) == gpu_lib.KMEANS_OK
    got = gpu_lib.kmeans_cross_entropy_grad(dloss, x, w, bad, got[1], ws=ws)
    assert gpu_lib.kmeans_device_status(ws) == gpu_lib.KMEANS_ERR_DEVICE_LABEL
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m", [130, 5000])
def test_ignored_rows_may_hold_anything(gpu_lib, dtype, m):
    x, w, labels, dloss = draw(m, 500, 64, dtype, 4, 0.5)
    clean = gpu_lib.kmeans_cross_entropy(x, w, labels)
    grads = gpu_lib.kmeans_cross_entropy_grad(dloss, x, w, labels, clean[1])
    gone = labels < 0
    x[gone] = float("nan")
    dloss[gone] = float("inf")
    lse = clean[1].clone()
    lse[gone] = float("nan")
    got = gpu_lib.kmeans_cross_entropy(x, w, labels)
    assert all(torch.equal(a, b) for a, b in zip(got, clean))
    got = gpu_lib.kmeans_cross_entropy_grad(dloss, x, w, labels, lse)
    assert all(torch.equal(a, b) for a, b in zip(got, grads))
    assert not got[0][gone].any()


@pytest.mark.parametrize("dtype", DTYPES)
def test_no_row_counts(gpu_lib, dtype):
    for m in (0, 3, 5000):
        x, w, labels, dloss = draw(m, 90, 24, dtype, 1, 1.1)
        loss, lse = gpu_lib.kmeans_cross_entropy(x, w, labels)
        dx, dw = gpu_lib.kmeans_cross_entropy_grad(dloss, x, w, labels, lse)
        assert loss.shape == (m,) and not any(bool(t.any()) for t in (loss, lse, dx, dw))


def test_a_row_that_is_not_finite_keeps_to_itself(gpu_lib):
    x, w, labels, _ = draw(300, 700, 64, torch.bfloat16, 8)
    want = gpu_lib.kmeans_cross_entropy(x, w, labels)
    x[17, 3] = float("nan")
    x[200] = float("inf")
    got = gpu_lib.kmeans_cross_entropy(x, w, labels)
    keep = torch.ones(300, dtype=torch.bool, device="cuda")
    keep[[17, 200]] = False
    assert all(torch.equal(a[keep], b[keep]) for a, b in zip(got, want))
    assert math.isnan(got[0][17].item()) and not math.isfinite(got[0][200].item())


@pytest.mark.parametrize("dtype", DTYPES)
def test_large_logits(gpu_lib, dtype):
    """Logits of some hundreds: exponentials of what is below the largest, and a loss near zero keeps its digits."""
    m, n, k = 100, 600, 128
    x, w, labels, dloss = draw(m, n, k, dtype, 9)
    x = (8 * w[labels].float() * k ** 0.5).to(dtype)
    loss, _ = check_forward(gpu_lib, x, w, labels, scale=4.0)
    assert bool((loss >= 0).all())
    check_grad(gpu_lib, dloss, x, w, labels, scale=4.0)


def test_gradient_against_differences(gpu_lib):
    m, n, k = 3, 11, 6
    x, w, labels, dloss = draw(m, n, k, torch.float16, 2)
    _, lse = gpu_lib.kmeans_cross_entropy(x, w, labels, scale=0.7)
    dx, dw = gpu_lib.kmeans_cross_entropy_grad(dloss, x, w, labels, lse, scale=0.7)
    h = 1e-4

    def value(xx, ww):
        z = 0.7 * (xx @ ww.t())
        return (dloss.double() * (torch.logsumexp(z, 1) - z.gather(1, labels[:, None])[:, 0])).sum()

    for t, grad in ((0, dx), (1, dw)):
        for i in range(grad.shape[0]):
            for j in range(k):
                args = [x.double(), w.double()]
                args[t][i, j] += h
                up = value(*args)
                args[t][i, j] -= 2 * h
                want = ((up - value(*args)) / (2 * h)).item()
                # two roundings to float16 of terms of up to dloss |w| (or |x|)
                assert abs(grad[i, j].item() - want) <= 2e-3 * dloss.max().item() * 4 + 1e-7


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("k", [40, 41])
def test_a_pitch_and_an_odd_start(gpu_lib, dtype, k):
    x, w, labels, dloss = draw(90, 300, k, dtype, 3, 0.1)
    wide = torch.full((90, 2 * k + 3), float("nan"), dtype=dtype, device="cuda")
    wide[:, 1:1 + k] = x
    a, b = (gpu_lib.kmeans_cross_entropy(v, w, labels) for v in (x, wide[:, 1:1 + k]))
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    a, b = (gpu_lib.kmeans_cross_entropy_grad(dloss, v, w, labels, a[1]) for v in (x, wide[:, 1:1 + k]))
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_only_what_is_needed(gpu_lib):
    x, w, labels, dloss = draw(200, 300, 64, torch.bfloat16, 3, 0.1)
    _, lse = gpu_lib.kmeans_cross_entropy(x, w, labels)
    dx, dw = gpu_lib.kmeans_cross_entropy_grad(dloss, x, w, labels, lse)
    one = gpu_lib.kmeans_cross_entropy_grad(dloss, x, w, labels, lse, need_dw=False)
    two = gpu_lib.kmeans_cross_entropy_grad(dloss, x, w, labels, lse, need_dx=False)
    assert torch.equal(one[0], dx) and one[1] is None and two[0] is None and torch.equal(two[1], dw)


def test_gradients_of_very_different_sizes_in_float16(gpu_lib):
    """dloss over 2^20: the power of two serves the largest, and the smallest keeps the digits that the bound says."""
    x, w, labels, dloss = draw(60, 2000, 64, torch.float16, 12)
    dloss = dloss * torch.exp2(-torch.arange(60, device="cuda") / 3.0)
    check_grad(gpu_lib, dloss, x, w, labels)


def test_a_starved_pipeline_is_reported_and_the_next_call_works(gpu_lib, monkeypatch):
    x, w, labels, dloss = draw(300, 400, 128, torch.bfloat16, 1)
    ws = gpu_lib.cross_entropy_workspace(gpu_lib.OP_CROSS_ENTROPY_GRAD, 300, 400, 128)
    want = gpu_lib.kmeans_cross_entropy(x, w, labels, ws=ws)
    monkeypatch.setenv("KMEANS_GB300_TEST_STARVE_PIPELINE", "1")
    gpu_lib.kmeans_cross_entropy(x, w, labels, ws=ws)
    assert gpu_lib.kmeans_device_status(ws) == gpu_lib.KMEANS_ERR_DEVICE_TIMEOUT
    gpu_lib.kmeans_cross_entropy_grad(dloss, x, w, labels, want[1], ws=ws)
    assert gpu_lib.kmeans_device_status(ws) == gpu_lib.KMEANS_ERR_DEVICE_TIMEOUT
    monkeypatch.delenv("KMEANS_GB300_TEST_STARVE_PIPELINE")
    got = gpu_lib.kmeans_cross_entropy(x, w, labels, ws=ws)
    assert gpu_lib.kmeans_device_status(ws) == gpu_lib.KMEANS_OK
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m", [5, 64, 300])
@pytest.mark.parametrize("first", [0, 128, 576])
def test_closed_classes_and_open_ones_far_below_zero(gpu_lib, m, first, dtype):
    """256 neighbouring classes closed by a weight of -inf (more than any part of the classes whose sums are formed
    together), the others' logits near -200: the reference of the closed parts must not count."""
    n, k = 1000, 48
    x, w, labels, _ = draw(m, n, k, dtype, 21)
    x[:, 0], x[:, 1] = 1.0, 1.0
    w[:, 0], w[:, 1] = 0.0, -200.0
    open_ = torch.ones(n, dtype=torch.bool, device="cuda")
    open_[first:first + 256] = False
    w[~open_, 0] = -math.inf
    labels = open_.nonzero()[:, 0][labels % int(open_.sum())]
    loss, lse = gpu_lib.kmeans_cross_entropy(x, w, labels)
    z, _, _, cut = plain(x, w[open_], labels % int(open_.sum()), 1.0)  # (the label's own logit is taken below)
    want_lse = torch.logsumexp(z, 1)
    want = want_lse - (x.double() * w[labels].double()).sum(1)
    off = cut + 2.0 ** -21 + z.abs().amax(1) * 2.0 ** -22
    assert bool(((lse.double() - want_lse).abs() <= off).all())
    assert bool(((loss.double() - want).abs() <= 2 * off).all())


@pytest.mark.parametrize("m", [5, 300])
def test_a_closed_label_and_no_open_class(gpu_lib, m):
    x, w, labels, _ = draw(m, 700, 16, torch.bfloat16, 22)
    x[:, 0] = 1.0
    w[:, 0] = 0.0
    w[labels[0], 0] = -math.inf
    loss, lse = gpu_lib.kmeans_cross_entropy(x, w, labels)
    gone = labels == labels[0]
    assert bool(torch.isinf(loss[gone]).all()) and bool((loss[gone] > 0).all())
    assert bool(torch.isfinite(lse).all()) and bool(torch.isfinite(loss[~gone]).all())
    w[:, 0] = -math.inf
    loss, lse = gpu_lib.kmeans_cross_entropy(x, w, labels)
    assert bool((lse == -math.inf).all()) and bool(loss.isnan().all())


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("m", [60, 5000])
def test_a_gradient_that_is_not_finite_keeps_to_its_row_of_dx(gpu_lib, m, bad):
    """float16's power of two goes by the largest finite gradient: the other rows' dx stays what it was, to the bit."""
    x, w, labels, dloss = draw(m, 2000, 64, torch.float16, 13)
    _, lse = gpu_lib.kmeans_cross_entropy(x, w, labels)
    top = int(dloss.argmax())
    row = (top + m // 2) % m
    clean, _ = gpu_lib.kmeans_cross_entropy_grad(dloss, x, w, labels, lse)
    dloss[row] = bad
    dx, _ = gpu_lib.kmeans_cross_entropy_grad(dloss, x, w, labels, lse)
    keep = torch.ones(m, dtype=torch.bool, device="cuda")
    keep[row] = False
    assert torch.equal(dx[keep], clean[keep]) and not bool(torch.isfinite(dx[row]).any())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,n,k", [(1, 500, 64), (24, 3000, 128), (70, 700, 72), (300, 2000, 64)])
def test_the_label_term_of_dx_is_rounded_once(gpu_lib, m, n, k, dtype):
    """A row's dz has one large term, its label's, whose rounding to 16 bits would be that of all of dx: it is a power
    of two there, and dx is rounded once.  2^-b is allowed on the other terms alone; the label's is within what its
    probability is (p rel / (1 - p)) and some float32 roundings.  A dz rounded as it stands is outside that."""
    g = torch.Generator(device="cuda")
    g.manual_seed(m)
    w = 0.05 * torch.randn(n, k, generator=g, device="cuda")
    labels = torch.randperm(n, generator=g, device="cuda")[:m]
    w[labels] *= 20.0
    w = w.to(dtype)
    x = (0.1 * torch.randn(m, k, generator=g, device="cuda")).to(dtype)
    dloss = 1.0 + torch.rand(m, generator=g, device="cuda")
    _, lse = gpu_lib.kmeans_cross_entropy(x, w, labels)
    dx, _ = gpu_lib.kmeans_cross_entropy_grad(dloss, x, w, labels, lse, need_dw=False)
    z, want_lse, _, cut = plain(x, w, labels, 1.0)
    gd, wd = dloss.double()[:, None], w.double()
    p = torch.exp(z - want_lse[:, None])
    hot = torch.nn.functional.one_hot(labels, n).double()
    dz = gd * (p - hot)
    rel = (2 * cut + 2.0 ** -20 + z.abs().amax(1) * 2.0 ** -21)[:, None]
    b = 2.0 ** -BITS[dtype]
    others = gd * p * (1 - hot) * (rel + b * (1 + rel)) + (2.0 ** -38 * dloss.max().item() if dtype is torch.float16 else 0)
    label = gd * hot * (p * rel + 2.0 ** -20 * (1 - p))
    off = (others + label) @ wd.abs() + (CUT * n + 2.0 ** -20) * (dz.abs() @ wd.abs())
    want = dz @ wd
    bound = off + 1.01 * b * (want.abs() + off) + TINY[dtype]
    assert bool(((dx.double() - want).abs() <= bound).all())
    rounded = (dz.to(dtype).double() @ wd).to(dtype).double()
    if m > 1:  # (one row's rounding may happen to be small)
        assert bool(((rounded - want).abs() > bound).any())

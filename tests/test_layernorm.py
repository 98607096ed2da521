"""Layer norm and its gradient on the GPU against float64.

Bounds, fixed before any run, with u = 2^-24 and a sum of d values added 32 to a
thread (d / 1024 where a row is longer than registers hold) and then in a tree
within e = (48 + d / 1024) u of its terms' magnitudes.  The mean is corrected by
a second sum about itself, which leaves e mean|x - mean| and half its last bit;
rstd is within (e + 4 u) of itself (2^-22 the reciprocal root's own).  A value
kept in b significant bits is within 2^-b of itself.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

BITS = {torch.float32: 24, torch.float16: 11, torch.bfloat16: 8}
TINY = {torch.float32: 0.0, torch.float16: 2.0 ** -25, torch.bfloat16: 0.0}
DTYPES = [torch.float32, torch.float16, torch.bfloat16]
U = 2.0 ** -24
EPS = 1e-5

SHAPES = [(0, 16), (1, 1), (1, 4096), (3, 8), (5, 33), (17, 64), (260, 65), (33, 512), (9, 1031), (64, 1024), (7, 2048),
          (5, 4095), (40, 4096), (6, 8192), (3, 8200), (2, 16384), (3, 20001), (2, 40000), (2, 70000), (1500, 24)]


def normal(shape, dtype, seed, scale=1.0, shift=0.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale + shift).to(dtype)


def err(d):
    return (48 + d / 1024) * U


def stats(x):
    x = x.double()
    mean = x.mean(1)
    var = (x - mean[:, None]).square().mean(1)
    return mean, var


def check_forward(km, x, w, b):
    (n, d), dtype = x.shape, x.dtype
    y, mean, rstd = km.kmeans_layernorm(x, w, b, eps=EPS, save_stats=True)
    mu, var = stats(x)
    rs = (var + EPS) ** -0.5
    off = x.double() - mu[:, None]
    e = err(d)
    mean_off = e * off.abs().mean(1) + U * mu.abs()
    assert bool(((mean.double() - mu).abs() <= mean_off).all())
    rel = e + 4 * U + 2.0 ** -22
    assert bool(((rstd.double() - rs).abs() <= rel * rs).all())
    wd = w.double() if w is not None else torch.ones((), device="cuda")
    bd = b.double() if b is not None else torch.zeros((), device="cuda")
    want = off * rs[:, None] * wd + bd
    # (x - mean is itself rounded, at the size of what is left)
    bound = ((e * off.abs().mean(1) * rs)[:, None] + (off * rs[:, None]).abs() * (rel + 6 * U)) * wd.abs() \
        + U * (want.abs() + bd.abs()) + 1.01 * 2.0 ** -BITS[dtype] * want.abs() + TINY[dtype]
    assert bool(((y.double() - want).abs() <= bound).all())


def check_grad(km, dy, x, w, res):
    (n, d), dtype = x.shape, x.dtype
    mu, var = stats(x)
    mean, rstd = mu.float(), ((var + EPS) ** -0.5).float()
    dx, dw, db = km.kmeans_layernorm_grad(dy, x, mean, rstd, weight=w, residual=res)
    dyd, rs = dy.double(), rstd.double()[:, None]
    h = (x.double() - mean.double()[:, None]) * rs
    g = dyd * w.double() if w is not None else dyd
    mg, mgh = g.mean(1, keepdim=True), (g * h).mean(1, keepdim=True)
    want = rs * (g - mg - h * mgh)
    e = err(d)
    size = rs * (e * g.abs().mean(1, keepdim=True) + (e + 4 * U) * h.abs() * (g * h).abs().mean(1, keepdim=True)
                 + 6 * U * (g.abs() + mg.abs() + (h * mgh).abs()))
    if res is not None:
        want, size = want + res.double(), size + U * res.double().abs()
    bound = size + 1.01 * 2.0 ** -BITS[dtype] * want.abs() + U * want.abs() + TINY[dtype]
    assert bool(((dx.double() - want).abs() <= bound).all())
    # a column's sum: up to n / 16 rows in a thread, the threads' in a tree
    terms = (n / 16 + 64) * U
    for got, part in ((dw, dyd * h), (db, dyd)):
        total = part.sum(0)
        limit = terms * part.abs().sum(0) + 1.01 * 2.0 ** -BITS[dtype] * total.abs() + TINY[dtype]
        assert bool(((got.double() - total).abs() <= limit).all())
    again = km.kmeans_layernorm_grad(dy, x, mean, rstd, weight=w, residual=res)
    assert all(torch.equal(p, q) for p, q in zip((dx, dw, db), again))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,d", SHAPES)
@pytest.mark.parametrize("affine,shift", [(True, 0.0), (False, 20.0)])
def test_rows_are_normalised(gpu_lib, n, d, dtype, affine, shift):
    w, b = (normal((d,), dtype, 1, 0.3, 1.0), normal((d,), dtype, 2)) if affine else (None, None)
    check_forward(gpu_lib, normal((n, d), dtype, d, shift=shift), w, b)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,d", SHAPES)
@pytest.mark.parametrize("affine,residual", [(True, True), (False, False)])
def test_gradient(gpu_lib, n, d, dtype, affine, residual):
    check_grad(gpu_lib, normal((n, d), dtype, d + 1), normal((n, d), dtype, d, shift=1.0),
               normal((d,), dtype, 1, 0.3, 1.0) if affine else None, normal((n, d), dtype, 3) if residual else None)


@pytest.mark.parametrize("d", [40, 4096, 4100])
def test_only_what_is_needed(gpu_lib, d):
    x, dy = normal((70, d), torch.bfloat16, 1), normal((70, d), torch.bfloat16, 2)
    _, mean, rstd = gpu_lib.kmeans_layernorm(x, save_stats=True)
    whole = gpu_lib.kmeans_layernorm_grad(dy, x, mean, rstd)
    for need in range(8):
        flags = [bool(need >> i & 1) for i in range(3)]
        got = gpu_lib.kmeans_layernorm_grad(dy, x, mean, rstd, need_dx=flags[0], need_dweight=flags[1],
                                            need_dbias=flags[2])
        for flag, a, b in zip(flags, got, whole):
            assert torch.equal(a, b) if flag else a is None


def test_no_rows_have_no_weight_gradient(gpu_lib):
    x = torch.zeros(0, 24, device="cuda")
    stat = torch.zeros(0, device="cuda")
    dx, dw, db = gpu_lib.kmeans_layernorm_grad(x, x, stat, stat, dweight=torch.full((24,), 7.0, device="cuda"))
    assert dx.shape == (0, 24) and not dw.any() and not db.any()


@pytest.mark.parametrize("dtype", DTYPES)
def test_gradient_against_differences(gpu_lib, dtype):
    n, d = 3, 20
    x, dy = normal((n, d), dtype, 1).double(), normal((n, d), dtype, 2).double()
    w = normal((d,), dtype, 3, 0.3, 1.0).double()

    def value(v):
        mu, var = stats(v)
        return (((v - mu[:, None]) * ((var + EPS) ** -0.5)[:, None] * w) * dy).sum(1)

    _, mean, rstd = gpu_lib.kmeans_layernorm(x.to(dtype), w.to(dtype), eps=EPS, save_stats=True)
    dx, _, _ = gpu_lib.kmeans_layernorm_grad(dy.to(dtype), x.to(dtype), mean, rstd, weight=w.to(dtype))
    h = 1e-5
    for j in range(d):
        step = torch.zeros_like(x)
        step[:, j] = h
        want = (value(x + step) - value(x - step)) / (2 * h)
        assert bool(((dx[:, j].double() - want).abs() <= 1e-4 + 2.0 ** -BITS[dtype] * 1.01 * want.abs()).all())


def test_large_offsets_keep_their_digits(gpu_lib):
    """Rows around 4096 in float32: the values hold the spread to 2^-12 of it, and the mean must not lose more."""
    x = normal((20, 3000), torch.float32, 5, shift=4096.0)
    y, mean, rstd = gpu_lib.kmeans_layernorm(x, save_stats=True)
    mu, var = stats(x)
    assert bool(((mean.double() - mu).abs() <= 2 * U * mu.abs()).all())
    want = (x.double() - mu[:, None]) * ((var + EPS) ** -0.5)[:, None]
    assert (y.double() - want).abs().max().item() < 2e-5


def test_equal_values_and_zero_eps(gpu_lib):
    x = torch.full((2, 1000), 3.7, device="cuda")
    y, mean, rstd = gpu_lib.kmeans_layernorm(x, eps=EPS, save_stats=True)
    assert (y.abs().max() <= 1e-3).item() and abs(mean[0].item() - 3.7) < 1e-6
    assert abs(rstd[0].item() * EPS ** 0.5 - 1) < 1e-3


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_what_is_not_finite_stays_in_its_row(gpu_lib, bad):
    x = normal((9, 100), torch.float32, 1)
    clean = gpu_lib.kmeans_layernorm(x, save_stats=True)
    x[4, 50] = bad
    got = gpu_lib.kmeans_layernorm(x, save_stats=True)
    keep = [r for r in range(9) if r != 4]
    for a, b in zip(clean, got):
        assert torch.equal(a[keep], b[keep])
    assert bool(got[0][4].isnan().all())
    dx, _, _ = gpu_lib.kmeans_layernorm_grad(x, x, got[1], got[2])
    assert bool(torch.isfinite(dx[keep]).all())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [61, 64, 1000])
def test_pitches_and_odd_starts(gpu_lib, dtype, d):
    big = normal((50, 3 * d + 7), dtype, 1)
    x, dy, res = big[:, 1:1 + d], big[:, d + 2:2 * d + 2], big[:, 2 * d + 3:3 * d + 3]
    wb = normal((2 * d + 1,), dtype, 2)
    w, b = wb[1:d + 1], wb[d + 1:]
    check_forward(gpu_lib, x, w, b)
    check_grad(gpu_lib, dy, x, w, res)


@pytest.mark.parametrize("d", [100, 4096, 4099, 40000])
def test_in_place(gpu_lib, d):
    x, dy, res = (normal((30, d), torch.bfloat16, s) for s in (1, 2, 3))
    want, mean, rstd = gpu_lib.kmeans_layernorm(x, save_stats=True)
    y = x.clone()
    assert gpu_lib.kmeans_layernorm(y, y=y)[0] is y and torch.equal(y, want)
    grads = gpu_lib.kmeans_layernorm_grad(dy, x, mean, rstd, residual=res)
    for at in ("dy", "residual"):
        a = {"dy": dy.clone(), "residual": res.clone()}
        got = gpu_lib.kmeans_layernorm_grad(a["dy"], x, mean, rstd, residual=a["residual"], dx=a[at])
        assert all(torch.equal(p, q) for p, q in zip(got, grads))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,d", [(1, 2), (5, 33), (17, 64), (9, 1031), (40, 4096), (3, 8200), (2, 40000)])
def test_no_eps_at_all(gpu_lib, n, d, dtype, monkeypatch):
    import sys
    monkeypatch.setattr(sys.modules[__name__], "EPS", 0.0)
    x = normal((n, d), dtype, d)
    check_forward(gpu_lib, x, normal((d,), dtype, 1, 0.3, 1.0), normal((d,), dtype, 2))
    check_grad(gpu_lib, normal((n, d), dtype, d + 1), x, normal((d,), dtype, 1, 0.3, 1.0), None)


@pytest.mark.parametrize("d", [8, 1024, 32768])
def test_equal_values_without_eps_are_not_finite_in_their_row_alone(gpu_lib, d):
    """0 / 0 by definition.  (Twos and a power of two of them: the mean is exact, and so is the variance.)"""
    x = normal((7, d), torch.float32, 1)
    clean = gpu_lib.kmeans_layernorm(x, eps=0.0, save_stats=True)
    x[3] = 2.0
    y, mean, rstd = gpu_lib.kmeans_layernorm(x, eps=0.0, save_stats=True)
    keep = [r for r in range(7) if r != 3]
    assert all(torch.equal(a[keep], b[keep]) for a, b in zip((y, mean, rstd), clean))
    assert mean[3].item() == 2.0 and rstd[3].item() == float("inf") and bool(y[3].isnan().all())
    dx, _, _ = gpu_lib.kmeans_layernorm_grad(x, x, mean, rstd, need_dweight=False, need_dbias=False)
    assert bool(torch.isfinite(dx[keep]).all()) and not bool(torch.isfinite(dx[3]).any())

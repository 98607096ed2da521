"""The gate and its gradient on the GPU against a plain implementation in
float64.

Bounds, fixed before any run.  The choice is exact.  An exponential of x <= 0 is
within |x| 2^-23 + 2^-22 of itself, a softmax's sum of E of them within (E / 128
+ 8) 2^-24 more, a quotient within 2^-22: a score is within (|x| + 6 + E / 512)
2^-22 of itself, x the logit's distance from the row's largest (from zero for the
logistic function), a renormalised weight within twice that.  A gradient's error
is that of its weights over the terms' magnitudes, and one rounding.
"""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

BITS = {torch.float32: 24, torch.float16: 11, torch.bfloat16: 8}
TINY = {torch.float32: 2.0 ** -126, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -126}
DTYPES = [torch.float32, torch.float16, torch.bfloat16]


def scores_of(z, kind):
    with np.errstate(invalid="ignore", over="ignore"):
        if kind == "sigmoid":
            return 1 / (1 + np.exp(-z))
        e = np.exp(z - z.max(1, keepdims=True))
        return np.nan_to_num(e / e.sum(1, keepdims=True), nan=0.0)  # (a token without open experts)


def plain_gate(z, topk, kind, bias=None, groups=1, topk_groups=None, renormalize=True, scale=1.0):
    """By definition, token by token, in float64 (no NaN)."""
    n, E = z.shape
    s = scores_of(z, kind)
    ids, w = np.full((n, topk), -1, np.int64), np.zeros((n, topk))
    size = E // groups
    for t in range(n):
        c = z[t].copy() if bias is None else s[t] + bias
        c[z[t] == -np.inf] = -np.inf
        if groups > 1:
            v = np.where(z[t] == -np.inf, -np.inf, s[t] + (0 if bias is None else bias))
            total = []
            for g in range(groups):
                best = sorted(v[g * size:(g + 1) * size], reverse=True)[:2]
                total.append(sum(b for b in best if b != -np.inf) if best[0] != -np.inf else -np.inf)
            order = sorted(range(groups), key=lambda g: (-total[g], g))
            for g in order[topk_groups:]:
                c[g * size:(g + 1) * size] = -np.inf
        order = sorted((e for e in range(E) if c[e] != -np.inf), key=lambda e: (-c[e], e))[:topk]
        ids[t, :len(order)] = order
        w[t, :len(order)] = s[t, order]
        if renormalize and order:
            w[t] /= w[t].sum()
    return ids, w * scale


def draw(n, E, dtype, seed, closed=0.0):
    r = np.random.RandomState(seed)
    z = torch.from_numpy(2 * r.randn(n, E)).to(dtype)
    z[torch.from_numpy(r.rand(n, E) < closed)] = -math.inf
    return z


def weight_bound(z, ids, kind, renormalize):
    top = z.max(1, keepdims=True)
    far = np.abs(z) if kind == "sigmoid" else np.abs(z - np.where(np.isfinite(top), top, 0))
    far = np.take_along_axis(far, np.maximum(ids, 0), 1)
    far = np.where(np.isfinite(far), far, 0)
    rel = (far + 6 + z.shape[1] / 512) * 2.0 ** -22
    return 2 * rel.max(1, keepdims=True, initial=0) if renormalize else rel


CASES = [  # n, E, topk, groups, topk_groups, closed
    (0, 8, 2, 1, 1, 0.0), (1, 1, 1, 1, 1, 0.0), (1, 64, 2, 1, 1, 0.0), (5, 2, 2, 2, 1, 0.0), (33, 7, 3, 1, 1, 0.3),
    (130, 33, 8, 3, 2, 0.1), (257, 64, 6, 8, 3, 0.0), (100, 96, 32, 4, 4, 0.2), (64, 256, 8, 8, 4, 0.0),
    (31, 257, 5, 1, 1, 0.5), (50, 1000, 10, 20, 7, 0.0), (9, 1024, 4, 32, 5, 0.9), (7, 4096, 32, 1, 1, 0.0),
    (6, 4095, 8, 9, 2, 0.0), (17, 12, 0, 1, 1, 0.0), (40, 16, 8, 4, 2, 1.0),
]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("n,E,topk,groups,topk_groups,closed", CASES)
@pytest.mark.parametrize("biased,renormalize,scale", [(False, True, 1.0), (True, False, 2.5), (True, True, 1.0)])
def test_choice_and_weights(gpu_lib, n, E, topk, groups, topk_groups, closed, kind, dtype, biased, renormalize, scale):
    z = draw(n, E, dtype, n + E, closed)
    bias = (0.1 * np.random.RandomState(E).randn(E)).astype(np.float32) if biased else None
    ids, w = gpu_lib.kmeans_gate(z.cuda(), topk, scores=kind, bias=None if bias is None else torch.from_numpy(bias).cuda(),
                                 groups=groups, topk_groups=topk_groups, renormalize=renormalize, scale=scale)
    assert ids.dtype == torch.int32 and w.dtype == torch.float32 and ids.shape == w.shape == (n, topk)
    z = z.double().numpy()
    want_ids, want = plain_gate(z, topk, kind, None if bias is None else bias.astype(np.float64), groups, topk_groups,
                                renormalize, scale)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    off = np.abs(w.cpu().double().numpy() - want)
    assert (off <= weight_bound(z, want_ids, kind, renormalize) * want + 2.0 ** -126).all()


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,topk_groups", [(1, 1), (8, 3)])
def test_sums_that_float32_cannot_tell_apart(gpu_lib, kind, groups, topk_groups):
    """A bias that cancels the scores: the order is decided by what the bias's own rounding leaves, some 2^-26."""
    n, E, topk = 60, 128, 9
    r = np.random.RandomState(4)
    z1 = r.randn(E).astype(np.float32)
    z = torch.from_numpy(np.repeat(z1[None], n, 0) + 1e-3 * r.randn(n, 1).astype(np.float32) * (kind == "softmax"))
    bias = (0.5 - scores_of(z[:1].double().numpy(), kind)[0]).astype(np.float32)
    ids, _ = gpu_lib.kmeans_gate(z.cuda(), topk, scores=kind, bias=torch.from_numpy(bias).cuda(), groups=groups,
                                 topk_groups=topk_groups)
    want, _ = plain_gate(z.double().numpy(), topk, kind, bias.astype(np.float64), groups, topk_groups)
    assert np.array_equal(ids.cpu().numpy(), want)


def near_case(kind, groups, topk_groups, n=1500, E=48, topk=9):
    """Scores and a bias that cancel to about 2^-25, differently for every token: some neighbours in the order are
    2^-32 apart, some less than 2^-38.  Returns also the smallest distance that decides anything."""
    r = np.random.RandomState(7)
    base = r.randn(E).astype(np.float32)
    bias = (0.5 - scores_of(base[None].astype(np.float64), kind)[0]).astype(np.float32)
    z = base * (1 + r.randint(-1, 2, (n, E)) * np.float32(2.0 ** -23))
    z = z.astype(np.float32)
    c = scores_of(z.astype(np.float64), kind) + bias
    least = []
    if groups > 1:
        size = E // groups
        total = np.sort(c.reshape(n, groups, size), 2)[:, :, -2:].sum(2)
        order = -np.sort(-total, 1)
        least.append(order[:, topk_groups - 1] - order[:, topk_groups])
        kept = total >= order[:, topk_groups - 1:topk_groups]
        c = np.where(np.repeat(kept, size, 1), c, -np.inf)
    order = -np.sort(-c, 1)[:, :topk + 1]
    least.append((order[:, :-1] - order[:, 1:]).ravel())
    return z, bias, np.concatenate(least)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,topk_groups", [(1, 1), (8, 3)])
def test_the_order_of_sums_that_are_nearer_and_nearer(gpu_lib, kind, groups, topk_groups):
    z, bias, gaps = near_case(kind, groups, topk_groups)
    # both ways of telling them apart are needed, and float64 itself (2^-52 of 1) is enough
    assert (gaps < 2.0 ** -38).sum() >= 5 and (gaps > 2.0 ** -38).sum() > 1000 and gaps.min() > 2.0 ** -50
    ids, _ = gpu_lib.kmeans_gate(torch.from_numpy(z).cuda(), 9, scores=kind, bias=torch.from_numpy(bias).cuda(),
                                 groups=groups, topk_groups=topk_groups)
    want, _ = plain_gate(z.astype(np.float64), 9, kind, bias.astype(np.float64), groups, topk_groups)
    assert np.array_equal(ids.cpu().numpy(), want)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_equal_experts_are_taken_by_index(gpu_lib, kind, biased):
    z = torch.zeros(3, 100)
    z[1, ::2] = -0.0
    z[2] = 1.0
    z[2, 50:] = 1.5
    bias = torch.full((100,), 0.25).cuda() if biased else None
    ids, w = gpu_lib.kmeans_gate(z.cuda(), 6, scores=kind, bias=bias)
    assert ids.tolist() == [[0, 1, 2, 3, 4, 5]] * 2 + [[50, 51, 52, 53, 54, 55]]
    assert torch.allclose(w, torch.full_like(w, 1 / 6), rtol=1e-6, atol=0)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_closed_experts(gpu_lib, kind):
    z = torch.full((4, 40), -math.inf)
    z[1, 7] = -300.0
    z[2, 3], z[2, 30] = -200.0, -201.0
    z[3, :] = 0.0
    bias = torch.zeros(40)
    bias[0] = -math.inf
    for b in (None, bias.cuda()):
        ids, w = gpu_lib.kmeans_gate(z.cuda(), 3, scores=kind, bias=b)
        assert ids[:3].tolist() == [[-1, -1, -1], [7, -1, -1], [3, 30, -1]]
        assert ids[3].tolist() == ([0, 1, 2] if b is None else [1, 2, 3])
        assert w[0].tolist() == [0, 0, 0] and w[1].tolist() == [1, 0, 0]
        e = math.exp(-1)
        assert abs(w[2, 0].item() - 1 / (1 + e)) < 1e-6 and abs(w[2, 1].item() - e / (1 + e)) < 1e-6


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
def test_a_nan_shows_and_stays_with_its_token(gpu_lib, kind, renormalize):
    z = draw(6, 50, torch.float32, 3)
    clean = gpu_lib.kmeans_gate(z.cuda(), 4, scores=kind, renormalize=renormalize)
    z[2, 31] = math.nan
    z[4, 8] = math.inf
    ids, w = gpu_lib.kmeans_gate(z.cuda(), 4, scores=kind, renormalize=renormalize)
    assert ids[2, 0].item() == 31 and math.isnan(w[2, 0].item()) and ids[4, 0].item() == 8
    if kind == "softmax":
        assert bool(w[2].isnan().all()) and bool(w[4].isnan().all())
    else:
        assert not bool(w[4].isnan().any())
    for t in (0, 1, 3, 5):
        assert torch.equal(ids[t], clean[0][t]) and torch.equal(w[t], clean[1][t])


def test_logits_with_a_pitch_and_an_odd_start(gpu_lib):
    z = draw(77, 200, torch.bfloat16, 9).cuda()
    want = gpu_lib.kmeans_gate(z[:, 3:100].contiguous(), 5)
    got = gpu_lib.kmeans_gate(z[:, 3:100], 5)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    dw = torch.randn(77, 5, device="cuda")
    assert torch.equal(gpu_lib.kmeans_gate_grad(dw, z[:, 3:100], want[0]),
                       gpu_lib.kmeans_gate_grad(dw, z[:, 3:100].contiguous(), want[0]))


# --------------------------------------------------------------- gradient
def plain_grad(dw, z, ids, kind, renormalize, scale):
    """From the Jacobian of the weights: (gradient, magnitude of its terms)."""
    n, E = z.shape
    s = scores_of(z, kind)
    dz, size = np.zeros((n, E)), np.zeros((n, E))
    for t in range(n):
        js = [j for j in range(ids.shape[1]) if 0 <= ids[t, j] < E and z[t, ids[t, j]] != -np.inf]
        at = ids[t, js]
        g, p = scale * dw[t, js], s[t, at]
        if not js:
            continue
        if renormalize:
            v = p / p.sum()
            ds, ds_size = v * (g - (g * v).sum()), v * (np.abs(g) + (np.abs(g) * v).sum())  # times the score
            if kind == "sigmoid":
                ds, ds_size = ds * (1 - p), ds_size * (1 - p)
            for k, e in enumerate(at):
                dz[t, e] += ds[k]
                size[t, e] += ds_size[k]
        elif kind == "sigmoid":
            for k, e in enumerate(at):
                dz[t, e] += g[k] * p[k] * (1 - p[k])
                size[t, e] += abs(g[k]) * p[k] * (1 - p[k])
        else:
            row, mag = np.zeros(E), np.zeros(E)
            for k, e in enumerate(at):
                row[e] += g[k]
                mag[e] += abs(g[k])
            dz[t] = s[t] * (row - (g * p).sum())
            size[t] = s[t] * (mag + (np.abs(g) * p).sum())
    return dz, size


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("n,E,topk,groups,topk_groups,closed", CASES)
def test_gradient(gpu_lib, n, E, topk, groups, topk_groups, closed, kind, dtype, renormalize):
    z = draw(n, E, dtype, n + E + 1, closed)
    r = np.random.RandomState(n)
    ids = np.array([r.permutation(E)[:topk] for _ in range(n)]).reshape(n, topk).astype(np.int32)
    ids[r.rand(n, topk) < 0.1] = -1
    dw = torch.from_numpy(r.randn(n, topk).astype(np.float32))
    got = gpu_lib.kmeans_gate_grad(dw.cuda(), z.cuda(), torch.from_numpy(ids).cuda(), scores=kind,
                                   renormalize=renormalize, scale=1.5,
                                   dlogits=torch.full((n, E), 7.0, dtype=dtype, device="cuda"))
    z = z.double().numpy()
    want, size = plain_grad(dw.double().numpy(), z, ids, kind, renormalize, 1.5)
    top = z.max(1, keepdims=True) if E else z
    far = np.abs(z) if kind == "sigmoid" else np.abs(z - np.where(np.isfinite(top), top, 0))
    far = np.where(np.isfinite(far), far, 0).max(1, keepdims=True, initial=0)
    bound = 4 * (far + 8 + E / 512 + topk) * 2.0 ** -22 * size + 2.0 ** -BITS[dtype] * np.abs(want) * 1.01 + TINY[dtype]
    off = np.abs(got.cpu().double().numpy() - want)
    assert (off <= bound).all()


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
def test_gradient_against_differences(gpu_lib, kind, renormalize):
    n, E, topk = 4, 24, 5
    z = draw(n, E, torch.float32, 11)
    ids, _ = gpu_lib.kmeans_gate(z.cuda(), topk, scores=kind, renormalize=renormalize, scale=2.0)
    dw = torch.randn(n, topk, generator=torch.Generator().manual_seed(1))
    got = gpu_lib.kmeans_gate_grad(dw.cuda(), z.cuda(), ids, scores=kind, renormalize=renormalize, scale=2.0)
    zd, at, h = z.double().numpy(), ids.cpu().numpy(), 1e-5

    def value(zz):
        s = scores_of(zz, kind)
        w = np.take_along_axis(s, at, 1)
        if renormalize:
            w = w / w.sum(1, keepdims=True)
        return 2.0 * (w * dw.double().numpy()).sum(1)

    for e in range(E):
        up, down = zd.copy(), zd.copy()
        up[:, e] += h
        down[:, e] -= h
        want = (value(up) - value(down)) / (2 * h)
        # the difference's own error: h^2 / 6 of a third derivative of a few dw, rounding 1e-16 / h
        assert np.abs(got[:, e].cpu().double().numpy() - want).max() < 2e-6 * np.abs(dw.numpy()).sum(1).max() + 1e-8


def test_an_expert_named_twice_gets_the_sum(gpu_lib):
    z = draw(3, 10, torch.float32, 2)
    ids = np.array([[4, 4, 4], [1, 2, 1], [-1, 9, 10]], np.int32)  # 10: no such expert
    dw = torch.randn(3, 3, generator=torch.Generator().manual_seed(3))
    for kind in ("softmax", "sigmoid"):
        for renormalize in (False, True):
            got = gpu_lib.kmeans_gate_grad(dw.cuda(), z.cuda(), torch.from_numpy(ids).cuda(), scores=kind,
                                           renormalize=renormalize)
            want, size = plain_grad(dw.double().numpy(), z.double().numpy(), ids, kind, renormalize, 1.0)
            assert (np.abs(got.cpu().double().numpy() - want) <= 40 * 2.0 ** -22 * size + 1e-30).all()


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_a_closed_expert_has_no_gradient(gpu_lib, kind):
    z = torch.zeros(2, 6)
    z[0, 3] = -math.inf
    z[1] = -math.inf
    ids = torch.tensor([[1, 3], [0, 5]], dtype=torch.int32)
    for renormalize in (False, True):
        got = gpu_lib.kmeans_gate_grad(torch.ones(2, 2).cuda(), z.cuda(), ids.cuda(), scores=kind,
                                       renormalize=renormalize)
        assert bool(torch.isfinite(got[0]).all()) and got[0, 3].item() == 0
        assert bool((got[1] == 0).all())


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("E,groups", [(256, 1), (256, 8), (1000, 5), (4096, 16)])
def test_rows_of_many_equal_logits(gpu_lib, kind, biased, E, groups):
    """Padding that a router sees: rows of zeros, of few different values, and of one large one."""
    z = torch.zeros(4, E)
    z[1] = (torch.arange(E) % 3).float()
    z[2, E // 2] = 5.0
    z[3, E - 40:] = 1.0
    bias = np.zeros(E, np.float32)
    bias[::7] = 0.125
    ids, _ = gpu_lib.kmeans_gate(z.cuda(), 12, scores=kind, bias=torch.from_numpy(bias).cuda() if biased else None,
                                 groups=groups, topk_groups=max(1, groups // 2))
    want, _ = plain_gate(z.double().numpy(), 12, kind, bias.astype(np.float64) if biased else None, groups,
                         max(1, groups // 2))
    if groups > 1:  # equal groups' sums may differ by a rounding of float64 in the plain form: compare the values
        got = np.take_along_axis(z.numpy(), ids.cpu().numpy().astype(np.int64), 1)
        assert np.array_equal(np.sort(got, 1), np.sort(np.take_along_axis(z.numpy(), want, 1), 1))
    else:
        assert np.array_equal(ids.cpu().numpy(), want)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups", [(50, 1), (50, 5), (200, 1), (200, 8), (1000, 4)])
def test_an_expert_that_its_bias_closes_stays_closed_beside_a_nan(gpu_lib, kind, E, groups):
    """A softmax with a NaN (or an infinity) in it is NaN throughout: the open experts count as infinite then, the
    closed ones as closed."""
    z = draw(6, E, torch.float32, 3)
    bias = torch.linspace(-0.1, 0.1, E)
    closed = torch.arange(E) % 5 == 1
    bias[closed] = -math.inf
    z[2, 7], z[3, 6], z[4, 12] = math.nan, math.nan, math.inf  # (expert 6 is one of the closed)
    z[5, 11] = math.inf  # (and so is 11)
    ids, w = gpu_lib.kmeans_gate(z.cuda(), 6, scores=kind, bias=bias.cuda(), groups=groups, topk_groups=max(1, groups // 2))
    assert bool((ids >= 0).all()) and not bool(closed[ids.cpu().long()].any())
    for row in ids.tolist():
        assert len(set(row)) == 6
    clean, _ = gpu_lib.kmeans_gate(z[:2].cuda(), 6, scores=kind, bias=bias.cuda(), groups=groups,
                                   topk_groups=max(1, groups // 2))
    assert torch.equal(ids[:2], clean)


@pytest.mark.parametrize("kind,reach", [("sigmoid", 12.0), ("sigmoid", 30.0), ("softmax", 6.0), ("softmax", 20.0)])
@pytest.mark.parametrize("groups,topk_groups", [(1, 1), (6, 2)])
def test_near_sums_of_logits_over_the_whole_range(gpu_lib, kind, reach, groups, topk_groups):
    """As above with logits from one end of the exponential's range to the other: the pairs' exponential decides what
    is 2^-38 apart or more."""
    r = np.random.RandomState(int(reach))
    n, E, topk = 1500, 48, 9
    base = (reach * (2 * r.rand(E) - 1)).astype(np.float32)
    bias = (0.5 - scores_of(base[None].astype(np.float64), kind)[0]).astype(np.float32)
    z = (base * (1 + r.randint(-1, 2, (n, E)) * np.float32(2.0 ** -23))).astype(np.float32)
    c = scores_of(z.astype(np.float64), kind) + bias
    order = -np.sort(-c, 1)[:, :topk + 1]
    clear = ((order[:, :-1] - order[:, 1:]) > 2.0 ** -48).all(1)
    if groups > 1:
        total = -np.sort(-np.sort(c.reshape(n, groups, -1), 2)[:, :, -2:].sum(2), 1)
        clear &= total[:, topk_groups - 1] - total[:, topk_groups] > 2.0 ** -48
        kept = np.sort(c.reshape(n, groups, -1), 2)[:, :, -2:].sum(2) >= total[:, topk_groups - 1:topk_groups]
        order = -np.sort(-np.where(np.repeat(kept, E // groups, 1), c, -np.inf), 1)[:, :topk + 1]
        clear &= ((order[:, :-1] - order[:, 1:]) > 2.0 ** -48).all(1)
    assert clear.sum() > n // 2
    ids, _ = gpu_lib.kmeans_gate(torch.from_numpy(z).cuda(), topk, scores=kind, bias=torch.from_numpy(bias).cuda(),
                                 groups=groups, topk_groups=topk_groups)
    want, _ = plain_gate(z.astype(np.float64), topk, kind, bias.astype(np.float64), groups, topk_groups)
    assert np.array_equal(ids.cpu().numpy()[clear], want[clear])

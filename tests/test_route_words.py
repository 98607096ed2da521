"""The row movers at every alignment that their words follow: stored rows on
16, 8, 4 or 2 bytes, the strided operand aligned otherwise, few and many
choices, and enough tokens for several words per thread.  Every tensor lies
between values that must survive (outputs) or must not be read into a result
(inputs: NaN).  Bounds as in test_route.py.
"""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from test_route import DTYPES, draw_ids, normal, plan, within  # noqa: E402

MARK = 123.0


class Placed:
    """A matrix `first` values into a buffer, rows `pitch` values apart, NaN or
    MARK everywhere else."""

    def __init__(self, rows, cols, dtype, first, pitch=None, values=None):
        pitch = pitch or cols
        fill = MARK if values is None else float("nan")
        self.flat = torch.full((first + rows * pitch + 64,), fill, dtype=dtype, device="cuda")
        self.t = self.flat[first:first + rows * pitch].view(rows, pitch)[:, :cols]
        if values is not None:
            self.t.copy_(values)
        self.first, self.size = first, rows * pitch

    def rest_is_untouched(self):
        return bool((self.flat[:self.first] == MARK).all()) and bool((self.flat[self.first + self.size:] == MARK).all())


def check(km, n, topk, n_experts, d, dtype, first, loose_first, loose_pitch, drop=0.1):
    ids = draw_ids(n, topk, n_experts, drop, seed=n + d + topk)
    offsets, order, rows = plan(km, ids, n_experts)
    kept = rows < offsets[-1]
    total = int(offsets[-1])
    t, j = kept.nonzero(as_tuple=True)
    x = Placed(n, d, dtype, loose_first, loose_pitch, normal((n, d), dtype, 1))
    xs, y, dys = (Placed(r, d, dtype, first) for r in (n * topk, n, n * topk))
    km.kmeans_route_gather(x.t, rows, offsets, xs=xs.t)
    want = torch.zeros(n * topk, d, dtype=dtype, device="cuda")
    want[:total] = x.t[order[:total].long() // topk]
    assert torch.equal(xs.t, want) and xs.rest_is_untouched()

    values = normal((n * topk, d), dtype, 2)
    values[total:] = float("nan")
    ys = Placed(n * topk, d, dtype, first, None, values)
    w = torch.rand(n, topk, device="cuda")
    km.kmeans_route_combine(ys.t, rows, offsets, weights=w, residual=x.t, y=y.t)
    part = torch.zeros(n, topk, d, dtype=torch.float64, device="cuda")
    part[kept] = ys.t[rows[kept].long()].double() * w[kept].double()[:, None]
    res = x.t.double()
    within(y.t, part.sum(1) + res, part.abs().sum(1) + res.abs(), topk + 1, dtype)
    assert y.rest_is_untouched()

    _, dw = km.kmeans_route_combine_grad(x.t, ys.t, rows, offsets, w, dys=dys.t)
    want = torch.zeros(n * topk, d, dtype=torch.float64, device="cuda")
    want[rows[t, j].long()] = w[t, j].double()[:, None] * res[t]
    within(dys.t, want, want.abs(), 1, dtype)
    assert dys.rest_is_untouched()
    prod = res[t] * ys.t[rows[t, j].long()].double()
    want_w, size = torch.zeros_like(w, dtype=torch.float64), torch.zeros_like(w, dtype=torch.float64)
    want_w[t, j], size[t, j] = prod.sum(1), prod.abs().sum(1)
    within(dw, want_w, size, d, torch.float32)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [2, 6, 7, 12, 36, 40, 154, 513])
@pytest.mark.parametrize("first", [0, 1, 2, 4])
@pytest.mark.parametrize("topk", [1, 3, 6])
def test_rows_at_any_alignment(gpu_lib, dtype, d, first, topk):
    # the strided operand aligned as the stored rows, better and worse
    for loose_first, loose_pitch in ((first, d), (0, (d + 7) // 8 * 8), (3, d + 5)):
        check(gpu_lib, 71, topk, 5, d, dtype, first, loose_first, loose_pitch)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("topk,d", [(1, 512), (2, 512), (2, 516), (3, 514), (5, 515)])
def test_enough_tokens_for_several_words_per_thread(gpu_lib, dtype, topk, d):
    check(gpu_lib, 21000, topk, 64, d, dtype, 0, 0, d)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [37, 38, 40])
def test_residual_is_the_output_at_any_alignment(gpu_lib, dtype, d):
    n, topk = 300, 3
    ids = draw_ids(n, topk, 7, 0.1, seed=d)
    offsets, _, rows = plan(gpu_lib, ids, 7)
    ys, x, w = normal((n * topk, d), dtype, 1), normal((n, d), dtype, 2), torch.rand(n, topk, device="cuda")
    for first in (0, 1, 2):
        apart = gpu_lib.kmeans_route_combine(ys, rows, offsets, weights=w, residual=x)
        same = Placed(n, d, dtype, first, None, x)
        gpu_lib.kmeans_route_combine(ys, rows, offsets, weights=w, residual=same.t, y=same.t)
        assert torch.equal(same.t, apart)

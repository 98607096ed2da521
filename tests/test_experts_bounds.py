"""The layer forward and back against float64, element by element.

The bound of every element follows the chain: each step's error is what its
operands bring, times the magnitudes they meet, and its own.  A product's sum of K
terms of magnitude S is within (K / 16 + 17) 2^-23 S, a float32 sum of T terms
within (T + 2) 2^-24 S, an activation or slope within 2^-19 (|z| + 1) and 1.2
times its argument's error, and what is kept in b bits within 2^-b of itself
(float16 also within 2^-25).  Products of two errors are left out: 2% more covers
them."""
import math

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

BITS = {torch.float16: 11, torch.bfloat16: 8}
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 0.0}


def normal(shape, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def gelu_tanh(z):
    return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))


def slope_of(z):
    z = z.clone().requires_grad_()
    out, = torch.autograd.grad(gelu_tanh(z).sum(), z)
    return out


class Bounded:
    """Values and how far they may be off."""

    def __init__(self, value, error=None):
        self.value, self.error = value, torch.zeros_like(value) if error is None else error

    def kept(self, dtype):
        return Bounded(self.value, self.error + 2.0 ** -BITS[dtype] * (self.value.abs() + self.error) + TINY[dtype])

    def plus(self, t):
        return Bounded(self.value + t, self.error)


def product(a, b, of=None):
    """a b^T with the tensor cores' cut-off; `of`: one more term's magnitude."""
    size = a.value.abs() @ b.value.abs().t()
    if of is not None:
        size = size + of.abs()
    error = a.error @ b.value.abs().t() + a.value.abs() @ b.error.t()
    return Bounded(a.value @ b.value.t(), error + (a.value.shape[1] / 16 + 17) * 2.0 ** -23 * size)


def check(name, got, want):
    off, bound = (got.double() - want.value).abs(), 1.02 * want.error
    assert bool((off <= bound).all()), f"{name}: off by {(off - bound).max().item():.3e} more than the bound"
    # and a result left out would be seen
    assert int((want.value != 0).sum()) < 64 or bool((want.value.abs() > bound).any()), name


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("n,topk,n_experts,d,hidden", [(1, 1, 4, 64, 96), (40, 2, 8, 72, 128), (600, 3, 6, 136, 256),
                                                       (1500, 1, 3, 200, 40)])
def test_every_element_of_the_layer(gpu_lib, n, topk, n_experts, d, hidden, dtype):
    from distance_argmin_gb300 import experts
    g = torch.Generator(device="cuda")
    g.manual_seed(n + topk)
    ids = torch.randint(0, n_experts, (n, topk), generator=g, device="cuda")
    if n > 1:
        ids[torch.rand(n, topk, generator=g, device="cuda") < 0.1] = -1
    x, res, dy = normal((n, d), dtype, 1), normal((n, d), dtype, 2), normal((n, d), dtype, 3)
    w1, w2 = normal((n_experts, hidden, d), dtype, 4, d ** -0.5), normal((n_experts, d, hidden), dtype, 5, hidden ** -0.5)
    b1, b2 = normal((n_experts, hidden), dtype, 6), normal((n_experts, d), dtype, 7)
    wts = torch.rand(n, topk, generator=g, device="cuda")
    y, saved = experts.experts_forward(x, ids, w1, w2, b1, b2, weights=wts, residual=res, activation="gelu_tanh",
                                       keep=True)
    grads = experts.experts_backward(dy, saved, w1, w2)

    zeros = lambda *s: torch.zeros(*s, dtype=torch.float64, device="cuda")
    out, out_size = Bounded(res.double(), zeros(n, d)), res.double().abs()
    dx, dx_size = Bounded(zeros(n, d)), zeros(n, d)
    dwts = Bounded(zeros(n, topk))
    for e in range(n_experts):
        t, j = (ids == e).nonzero(as_tuple=True)
        xe, w1e, w2e = Bounded(x[t].double()), Bounded(w1[e].double()), Bounded(w2[e].double())
        z = product(xe, w1e, b1[e].double()).plus(b1[e].double())
        near = 2.0 ** -19 * (z.value.abs() + 1)
        h = Bounded(gelu_tanh(z.value), 1.2 * z.error + near).kept(dtype)
        ys = product(h, w2e, b2[e].double()).plus(b2[e].double()).kept(dtype)
        wt = wts[t, j].double()[:, None]
        out.value.index_add_(0, t, wt * ys.value)
        out.error.index_add_(0, t, wt * ys.error)
        out_size.index_add_(0, t, wt * ys.value.abs())

        dyt = dy[t].double()
        dwts.value[t, j] = (dyt * ys.value).sum(1)
        dwts.error[t, j] = (dyt.abs() * (ys.error + (d + 2) * 2.0 ** -24 * ys.value.abs())).sum(1)
        dys = Bounded(wt * dyt, 2.0 ** -24 * (wt * dyt).abs()).kept(dtype)
        turned = lambda b: Bounded(b.value.t(), b.error.t())
        check(f"w2[{e}]", grads["w2"][e], product(turned(dys), turned(h)).kept(dtype))
        rows = t.numel()
        check(f"b2[{e}]", grads["b2"][e], Bounded(dys.value.sum(0), (dys.error + (rows + 2) * 2.0 ** -24
                                                                      * dys.value.abs()).sum(0)).kept(dtype))
        dh = product(dys, turned(w2e)).kept(dtype)
        pre = z.kept(dtype)
        s = slope_of(z.value)
        dz = Bounded(dh.value * s, dh.error * s.abs() + dh.value.abs() * (1.2 * pre.error + near))
        check(f"b1[{e}]", grads["b1"][e], Bounded(dz.value.sum(0), (dz.error + (rows + 2) * 2.0 ** -24
                                                                      * dz.value.abs()).sum(0)).kept(dtype))
        dz = dz.kept(dtype)
        check(f"w1[{e}]", grads["w1"][e], product(turned(dz), turned(xe)).kept(dtype))
        dxs = product(dz, turned(w1e)).kept(dtype)
        dx.value.index_add_(0, t, dxs.value)
        dx.error.index_add_(0, t, dxs.error)
        dx_size.index_add_(0, t, dxs.value.abs())
    out.error += (topk + 3) * 2.0 ** -24 * out_size
    dx.error += (topk + 2) * 2.0 ** -24 * dx_size
    check("y", y, out.kept(dtype))
    check("x", grads["x"], dx.kept(dtype))
    check("weights", grads["weights"], dwts)

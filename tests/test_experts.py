"""The expert layer on the GPU: the whole chain forward and back against float64,
and the example that trains and serves it.

Bound of the chain: every kept intermediate (hidden values, their gradients,
the experts' rows) is rounded to 16 bits of b significant bits once; with k and
h terms summed after each, the chain stays within 4 roundings 2^-b of the sums
of its terms' magnitudes.
"""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

BITS = {torch.float16: 11, torch.bfloat16: 8}


def normal(shape, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("n,topk,n_experts,d,hidden", [(1, 1, 4, 64, 96), (40, 2, 8, 72, 128), (600, 3, 6, 136, 256)])
def test_forward_and_gradient_of_the_layer(gpu_lib, n, topk, n_experts, d, hidden, dtype):
    from distance_argmin_gb300 import experts
    g = torch.Generator(device="cuda")
    g.manual_seed(n)
    ids = torch.randint(0, n_experts, (n, topk), generator=g, device="cuda")
    ids[torch.rand(n, topk, generator=g, device="cuda") < 0.1] = -1
    x, res, dy = normal((n, d), dtype, 1), normal((n, d), dtype, 2), normal((n, d), dtype, 3)
    w1, w2 = normal((n_experts, hidden, d), dtype, 4, d ** -0.5), normal((n_experts, d, hidden), dtype, 5, hidden ** -0.5)
    b1, b2 = normal((n_experts, hidden), dtype, 6), normal((n_experts, d), dtype, 7)
    wts = torch.rand(n, topk, generator=g, device="cuda")
    y, saved = experts.experts_forward(x, ids, w1, w2, b1, b2, weights=wts, residual=res, activation="gelu_tanh",
                                       keep=True)
    grads = experts.experts_backward(dy, saved, w1, w2)

    args = {"x": x, "w1": w1, "b1": b1, "w2": w2, "b2": b2, "weights": wts}
    args = {k: v.double().requires_grad_() for k, v in args.items()}

    def layer(a):
        out = res.double()
        for j in range(topk):
            for e in range(n_experts):
                t = (ids[:, j] == e).nonzero()[:, 0]
                z = a["x"][t] @ a["w1"][e].t() + a["b1"][e]
                h = torch.nn.functional.gelu(z, approximate="tanh")
                out = out.index_add(0, t, a["weights"][t, j, None] * (h @ a["w2"][e].t() + a["b2"][e]))
        return out

    want = layer(args)
    want.backward(dy.double())
    # the same sums over magnitudes bound what the roundings can do
    size = {k: v.detach().abs() for k, v in args.items()}

    def close(got, exact, name):
        unit = 4 * 2.0 ** -BITS[dtype]
        scale = exact.abs().max().clamp(min=1.0) if exact.numel() else 1.0
        assert bool(((got.double() - exact).abs() <= unit * (exact.abs() + scale)).all()), name

    assert all(torch.isfinite(v).all() for v in size.values())
    close(y, want.detach(), "y")
    for name, a in args.items():
        close(grads[name], a.grad, name)


def test_tokens_of_the_nearest_centroid(gpu_lib):
    from distance_argmin_gb300 import experts
    C = normal((16, 64), torch.float32, 1, 3.0)
    x = C[torch.arange(100, device="cuda") % 16] + normal((100, 64), torch.float32, 2, 0.1)
    ids = experts.nearest_experts(x, C)
    assert torch.equal(ids[:, 0], torch.arange(100, device="cuda") % 16)
    for n in (0, 1, 5, 15):
        assert torch.equal(experts.few_nearest_experts(x[:n].contiguous(), C), ids[:n])


def test_the_example_learns_and_serves(gpu_lib):
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import cluster_experts
    losses, served = cluster_experts.main(steps=40, n=4096, clusters=16)
    assert losses[-1] < 0.5 * losses[0]
    assert served < 2.0 * losses[-1]

"""The gradients of an expert block, expert by expert: each expert's matrices are
held to their own magnitude, also where one expert's are a small part of the
largest.

Bound: a row's gradient passes a rounding to 16 bits of b significant bits after
the loss, the output's, the combine's gradient and the second product's, and the
matrices' gradients one more; what the forward pass kept (normalised rows, hidden
values, the experts' outputs) was rounded once each.  Each is relative to the row
or the matrix it belongs to, and no step mixes experts, so that 12 roundings 2^-b
of the largest magnitude of an expert's own gradient bound its error.
"""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

BITS = {torch.float16: 11, torch.bfloat16: 8}


def normal(shape, dtype, seed, scale=1.0, shift=0.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale + shift).to(dtype)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("scores,renormalize", [("softmax", True), ("softmax", False), ("sigmoid", True)])
@pytest.mark.parametrize("n,topk,E,d,hidden", [(300, 2, 6, 64, 96), (90, 3, 8, 72, 40)])
def test_each_expert_by_its_own_magnitude(gpu_lib, n, topk, E, d, hidden, scores, renormalize, dtype):
    from distance_argmin_gb300 import experts
    x = normal((n, d), dtype, 1)
    gate_w, dy = normal((E, d), dtype, 2, d ** -0.5), normal((n, d), dtype, 3)
    w1, b1 = normal((E, hidden, d), dtype, 4, d ** -0.5), normal((E, hidden), dtype, 5, 0.1)
    w2, b2 = normal((E, d, hidden), dtype, 6, hidden ** -0.5), normal((E, d), dtype, 7, 0.1)
    w2[1], w1[2] = w2[1] / 16, w1[2] / 16  # one expert whose w1, one whose w2 has a small gradient
    y, saved = experts.block_forward(x, gate_w, w1, w2, topk, b1=b1, b2=b2, scores=scores, renormalize=renormalize,
                                     activation="silu", keep=True)
    got = experts.block_backward(dy, saved, gate_w, w1, w2)
    a = {k: v.double().requires_grad_() for k, v in dict(w1=w1, b1=b1, w2=w2, b2=b2).items()}
    xd = x.double()
    off = xd - xd.mean(1, keepdim=True)
    h = off * (off.square().mean(1, keepdim=True) + 1e-5) ** -0.5
    l = h @ gate_w.double().t()
    s = torch.softmax(l, 1) if scores == "softmax" else torch.sigmoid(l)
    ids = saved.ids.long()
    weights = s.gather(1, ids)
    if renormalize:
        weights = weights / weights.sum(1, keepdim=True)
    out = xd
    for j in range(topk):
        for e in range(E):
            t = (ids[:, j] == e).nonzero()[:, 0]
            hid = torch.nn.functional.silu(h[t] @ a["w1"][e].t() + a["b1"][e])
            out = out.index_add(0, t, weights[t, j, None] * (hid @ a["w2"][e].t() + a["b2"][e]))
    out.backward(dy.double())
    for name, v in a.items():
        for e in range(E):
            largest = v.grad[e].abs().max()
            assert largest > 0
            assert bool((got[name][e].double() - v.grad[e]).abs().max() <= 12 * 2.0 ** -BITS[dtype] * largest), (name, e)

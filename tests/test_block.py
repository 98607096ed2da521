"""The gate, the layer norm and the cross entropy together with the experts: a
block of a model and its loss, forward and back, against float64.

Bound: the choice of experts is taken over from the run (it is tested by itself);
every kept intermediate is rounded to 16 bits of b significant bits once.  A
gradient passes five of them on its longest way (dx of the loss, of the output
norm, of the experts' two products, of the gate's product), each a sum whose
roundings are its terms' own, so that they meet as their squares do; with what
the forward pass kept before them, 12 roundings 2^-b of the largest magnitude of
each result bound it.
"""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

BITS = {torch.float16: 11, torch.bfloat16: 8}


def normal(shape, dtype, seed, scale=1.0, shift=0.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale + shift).to(dtype)


def norm64(x, w, b, eps=1e-5):
    off = x - x.mean(1, keepdim=True)
    return off * (off.square().mean(1, keepdim=True) + eps) ** -0.5 * w + b


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("n,topk,E,d,hidden,classes,scores,renormalize", [
    (1, 1, 4, 64, 96, 50, "softmax", True), (50, 2, 8, 72, 128, 300, "softmax", False),
    (400, 3, 16, 136, 256, 1000, "sigmoid", True), (77, 2, 6, 65, 40, 129, "sigmoid", False)])
def test_a_block_and_its_loss(gpu_lib, n, topk, E, d, hidden, classes, scores, renormalize, dtype):
    from distance_argmin_gb300 import experts
    x = normal((n, d), dtype, 1)
    p = {"gate_w": normal((E, d), dtype, 2, d ** -0.5), "w1": normal((E, hidden, d), dtype, 3, d ** -0.5),
         "b1": normal((E, hidden), dtype, 4, 0.1), "w2": normal((E, d, hidden), dtype, 5, hidden ** -0.5),
         "b2": normal((E, d), dtype, 6, 0.1), "norm_weight": normal((d,), dtype, 7, 0.1, 1.0),
         "norm_bias": normal((d,), dtype, 8, 0.1), "out_w": normal((d,), dtype, 9, 0.1, 1.0),
         "out_b": normal((d,), dtype, 10, 0.1), "classes": normal((classes, d), dtype, 11, d ** -0.5)}
    bias = normal((E,), torch.float32, 12, 0.05)
    labels = torch.randint(0, classes, (n,), device="cuda", generator=torch.Generator(device="cuda").manual_seed(n))
    if n > 1:
        labels[::5] = -1
    how = dict(gate_bias=bias, scores=scores, renormalize=renormalize, scale=1.5, activation="gelu_tanh")
    y, saved = experts.block_forward(x, p["gate_w"], p["w1"], p["w2"], topk, p["norm_weight"], p["norm_bias"], p["b1"],
                                     p["b2"], keep=True, **how)
    served, none = experts.block_forward(x, p["gate_w"], p["w1"], p["w2"], topk, p["norm_weight"], p["norm_bias"], p["b1"],
                                         p["b2"], **how)
    assert none is None and torch.equal(served, y)
    z, mean, rstd = gpu_lib.kmeans_layernorm(y, p["out_w"], p["out_b"], save_stats=True)
    loss, lse = gpu_lib.kmeans_cross_entropy(z, p["classes"], labels)
    dloss = (labels >= 0).float()
    dz, dclasses = gpu_lib.kmeans_cross_entropy_grad(dloss, z, p["classes"], labels, lse)
    dy, dow, dob = gpu_lib.kmeans_layernorm_grad(dz, y, mean, rstd, weight=p["out_w"])
    grads = experts.block_backward(dy, saved, p["gate_w"], p["w1"], p["w2"], p["norm_weight"])
    grads.update(out_w=dow, out_b=dob, classes=dclasses)

    a = {k: v.double().requires_grad_() for k, v in p.items()}
    xd = x.double().requires_grad_()
    h = norm64(xd, a["norm_weight"], a["norm_bias"])
    l = h @ a["gate_w"].t()
    s = torch.softmax(l, 1) if scores == "softmax" else torch.sigmoid(l)
    ids = saved.ids.long()
    wts = s.gather(1, ids)
    if renormalize:
        wts = wts / wts.sum(1, keepdim=True)
    out = xd
    for j in range(topk):
        for e in range(E):
            t = (ids[:, j] == e).nonzero()[:, 0]
            hid = torch.nn.functional.gelu(h[t] @ a["w1"][e].t() + a["b1"][e], approximate="tanh")
            out = out.index_add(0, t, 1.5 * wts[t, j, None] * (hid @ a["w2"][e].t() + a["b2"][e]))
    logits = norm64(out, a["out_w"], a["out_b"]) @ a["classes"].t()
    live = labels >= 0
    want = (torch.logsumexp(logits, 1) - logits.gather(1, labels.clamp(min=0)[:, None])[:, 0]) * live
    want.sum().backward()

    def close(got, exact, name):
        unit = 12 * 2.0 ** -BITS[dtype]
        scale = exact.abs().max().clamp(min=1e-3) if exact.numel() else 1.0
        assert bool(((got.double() - exact).abs() <= unit * scale).all()), name

    close(y, out.detach(), "y")
    close(loss, want.detach(), "loss")
    close(grads["x"], xd.grad, "x")
    for name, v in a.items():
        close(grads[name], v.grad, name)


def test_a_block_without_a_norm_weight_and_on_a_stream(gpu_lib):
    from distance_argmin_gb300 import experts
    x, gw = normal((60, 64), torch.bfloat16, 1), normal((4, 64), torch.bfloat16, 2, 0.125)
    w1, w2 = normal((4, 96, 64), torch.bfloat16, 3, 0.125), normal((4, 64, 96), torch.bfloat16, 4, 0.1)
    y, saved = experts.block_forward(x, gw, w1, w2, 2, keep=True)
    grads = experts.block_backward(y, saved, gw, w1, w2)
    assert grads["norm_weight"] is None and grads["b1"] is None and grads["x"].shape == x.shape
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y2, saved2 = experts.block_forward(x, gw, w1, w2, 2, keep=True, stream=s)
    grads2 = experts.block_backward(y2, saved2, gw, w1, w2, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and all(torch.equal(a, grads2[k]) for k, a in grads.items() if a is not None)


def test_the_example_runs(gpu_lib):
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import gated_block
    losses, served = gated_block.main(steps=6, n=512, d=64, hidden=96, classes=300)
    assert len(losses) == 6 and all(v == v and v >= 0 for v in losses) and served == served


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_a_norm_with_a_bias_alone_or_a_weight_alone(gpu_lib, dtype):
    """The same as with the other one given as ones, or zeros."""
    from distance_argmin_gb300 import experts
    x, gw = normal((60, 64), dtype, 1), normal((4, 64), dtype, 2, 0.125)
    w1, w2 = normal((4, 96, 64), dtype, 3, 0.125), normal((4, 64, 96), dtype, 4, 0.1)
    weight, bias, dy = normal((64,), dtype, 5, 0.1, 1.0), normal((64,), dtype, 6, 0.1), normal((60, 64), dtype, 7)
    ones, zeros = torch.ones_like(weight), torch.zeros_like(bias)

    def both(norm_weight, norm_bias):
        y, saved = experts.block_forward(x, gw, w1, w2, 2, norm_weight, norm_bias, keep=True)
        return y, experts.block_backward(dy, saved, gw, w1, w2, norm_weight)

    for given, full, name in (((None, bias), (ones, bias), "norm_bias"), ((weight, None), (weight, zeros), "norm_weight")):
        (y, got), (want_y, want) = both(*given), both(*full)
        other = {"norm_bias": "norm_weight", "norm_weight": "norm_bias"}[name]
        assert torch.equal(y, want_y) and got[other] is None and got[name] is not None
        for key in ("x", "gate_w", "w1", "w2", name):
            assert torch.equal(got[key], want[key]), key


def test_a_norm_weight_that_the_forward_pass_did_not_have_is_refused(gpu_lib):
    from distance_argmin_gb300 import experts
    x, gw = normal((8, 64), torch.bfloat16, 1), normal((4, 64), torch.bfloat16, 2, 0.125)
    w1, w2 = normal((4, 32, 64), torch.bfloat16, 3, 0.125), normal((4, 64, 32), torch.bfloat16, 4, 0.1)
    weight = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    _, without = experts.block_forward(x, gw, w1, w2, 2, keep=True)
    _, having = experts.block_forward(x, gw, w1, w2, 2, weight, keep=True)
    for saved, norm_weight in ((without, weight), (having, None)):
        with pytest.raises(ValueError, match="norm_weight"):
            experts.block_backward(x, saved, gw, w1, w2, norm_weight)

"""A small model that classifies tokens: a block of gated experts and the cross
entropy of its output against the classes, trained and then served.

    python examples/gated_block.py [steps]

Every token is a noisy copy of the vector of its class, turned by the rotation of
its kind; the router learns which expert undoes which rotation, with a bias that
keeps the experts evenly loaded, and the classes' logits are never stored.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import distance_argmin_gb300 as km  # noqa: E402
from distance_argmin_gb300 import experts  # noqa: E402


def main(steps=80, n=4096, d=128, hidden=256, n_experts=8, topk=2, classes=5000, rate=0.01, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * scale

    kinds = normal(4, d, scale=1.0)
    turn = torch.linalg.qr(normal(4, d, d)).Q
    words = normal(classes, d)

    def batch(count):
        label = torch.randint(classes, (count,), generator=g, device="cuda")
        kind = torch.randint(4, (count,), generator=g, device="cuda")
        x = torch.bmm(turn[kind], words[label][:, :, None])[:, :, 0] + kinds[kind] + normal(count, d, scale=0.1)
        label[torch.rand(count, generator=g, device="cuda") < 0.1] = -1  # tokens that do not count
        return x.bfloat16(), label

    # fp32 copies are what the steps (Adam's) add to; the products take their bf16 values
    master = {"gate_w": normal(n_experts, d, scale=d ** -0.5), "w1": normal(n_experts, hidden, d, scale=d ** -0.5),
              "w2": normal(n_experts, d, hidden, scale=hidden ** -0.5), "norm_weight": torch.ones(d, device="cuda"),
              "norm_bias": torch.zeros(d, device="cuda"), "out_weight": torch.ones(d, device="cuda"),
              "out_bias": torch.zeros(d, device="cuda"), "classes": normal(classes, d, scale=d ** -0.5)}
    moments = {name: (torch.zeros_like(v), torch.zeros_like(v)) for name, v in master.items()}
    balance = torch.zeros(n_experts, device="cuda")

    def forward(p, x, keep):
        y, saved = experts.block_forward(x, p["gate_w"], p["w1"], p["w2"], topk, p["norm_weight"], p["norm_bias"],
                                         gate_bias=balance, keep=keep)
        z, mean, rstd = km.kmeans_layernorm(y, p["out_weight"], p["out_bias"], save_stats=keep)
        return y, saved, z, mean, rstd

    losses = []
    for step in range(1, steps + 1):
        p = {name: v.bfloat16() for name, v in master.items()}
        x, label = batch(n)
        y, saved, z, mean, rstd = forward(p, x, True)
        loss, lse = km.kmeans_cross_entropy(z, p["classes"], label, scale=2.0)
        counted = (label >= 0).sum()
        losses.append((loss.sum() / counted).item())
        dloss = (label >= 0).float() / counted
        dz, dclasses = km.kmeans_cross_entropy_grad(dloss, z, p["classes"], label, lse, scale=2.0)
        dy, dow, dob = km.kmeans_layernorm_grad(dz, y, mean, rstd, weight=p["out_weight"])
        grads = experts.block_backward(dy, saved, p["gate_w"], p["w1"], p["w2"], p["norm_weight"])
        grads.update(classes=dclasses, out_weight=dow, out_bias=dob)
        # experts with more than their part of the tokens get a lower bias, the others a higher one
        load = saved.offsets.diff().float()
        balance += 0.01 * torch.sign(load.mean() - load)
        for name, v in master.items():
            a, b = moments[name]
            grad = grads[name].float()
            a.lerp_(grad, 0.1)
            b.lerp_(grad * grad, 0.02)
            v -= rate * (a / (1 - 0.9 ** step)) / ((b / (1 - 0.98 ** step)).sqrt() + 1e-8)
    p = {name: v.bfloat16() for name, v in master.items()}

    # serving: one token at a time, as a decoding loop would
    x, label = batch(32)
    score = 0.0
    for t in range(x.shape[0]):
        _, _, z, _, _ = forward(p, x[t:t + 1].contiguous(), False)
        loss, _ = km.kmeans_cross_entropy(z, p["classes"], label[t:t + 1].contiguous(), scale=2.0)
        score += loss.item() / max(1, int((label >= 0).sum()))
    return losses, score


if __name__ == "__main__":
    losses, served = main(*(int(a) for a in sys.argv[1:2]))
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} in {len(losses)} steps, {served:.4f} served token by token")

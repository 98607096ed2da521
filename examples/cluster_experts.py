"""A layer of experts routed by k-means, trained and then served token by token.

    python examples/cluster_experts.py [steps]

Tokens drawn around 32 centers follow a different rotation in every cluster.
k-means finds the clusters, each becomes the domain of one expert, and the
experts learn the rotations by gradient steps; at the end single tokens are
answered one at a time.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import distance_argmin_gb300 as km  # noqa: E402
from distance_argmin_gb300 import experts  # noqa: E402


def main(steps=60, n=8192, d=256, hidden=512, clusters=32, rate=0.06, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * scale

    centers = normal(clusters, d, scale=3.0)
    turn = torch.linalg.qr(normal(clusters, d, d)).Q

    def batch(count):
        which = torch.randint(clusters, (count,), generator=g, device="cuda")
        x = centers[which] + normal(count, d, scale=0.5)
        y = torch.bmm(turn[which], ((x - centers[which]) * 2)[:, :, None])[:, :, 0]
        return x, y

    sample, _ = batch(n)
    C, *_ = km.kmeans_fit(sample, k=clusters, seed=seed)

    # fp32 copies are what the steps add to; the products take their bf16 values
    master = {"w1": normal(clusters, hidden, d, scale=d ** -0.5), "b1": torch.zeros(clusters, hidden, device="cuda"),
              "w2": normal(clusters, d, hidden, scale=hidden ** -0.5), "b2": torch.zeros(clusters, d, device="cuda")}
    losses = []
    for _ in range(steps):
        p = {name: v.bfloat16() for name, v in master.items()}
        x, target = batch(n)
        ids = experts.nearest_experts(x, C)
        xb = (x - C[ids[:, 0]]).bfloat16()
        y, saved = experts.experts_forward(xb, ids, p["w1"], p["w2"], p["b1"], p["b2"], keep=True)
        off = y.float() - target
        losses.append(off.square().mean().item())
        grads = experts.experts_backward((off * (2.0 * clusters / n)).bfloat16(), saved, p["w1"], p["w2"])
        for name, v in master.items():
            v -= rate * grads[name].float()
    p = {name: v.bfloat16() for name, v in master.items()}

    # serving: one token at a time, as a decoding loop would
    x, target = batch(64)
    off = 0.0
    for t in range(x.shape[0]):
        token = x[t:t + 1].contiguous()
        ids = experts.few_nearest_experts(token, C)
        y, _ = experts.experts_forward((token - C[ids[:, 0]]).bfloat16(), ids, p["w1"], p["w2"], p["b1"], p["b2"])
        off += (y.float() - target[t]).square().mean().item() / x.shape[0]
    return losses, off


if __name__ == "__main__":
    losses, served = main(*(int(a) for a in sys.argv[1:2]))
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} in {len(losses)} steps, {served:.4f} served token by token")

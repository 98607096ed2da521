"""A layer of experts: two products per expert, each token through the experts
it was sent to.

Which expert a token goes to is a choice of up to ``ROUTE_MAX_TOPK`` ids per
token.  With centroids it is the nearest one (``kmeans_assign``, the page "Three
shapes that fit an eager Gram assignment", section "Gram assignment"): the
clusters of the tokens are the experts, and a fit of the centroids on a sample
of tokens is all the training the choice needs.  A learned choice is a router's
(``kmeans_gate``), and ``block_forward`` is a whole block of a model around it:
layer norm, gate, experts and the residual stream.

    offsets, order, rows = kmeans_route(ids)            slots sorted by expert
    xs = kmeans_route_gather(x, rows, offsets)          tokens in that order
    h  = act(xs w1[e]^T + b1[e])                        kmeans_linear
    ys = h w2[e]^T + b2[e]                              kmeans_linear
    y[t] = residual[t] + sum_j weights[t, j] ys[rows[t, j]]   kmeans_route_combine

This module holds no arithmetic: it calls the C ABI through the binding in
order and keeps what the gradient needs.
"""
from __future__ import annotations

import functools


def _on_stream(fn):
    """Run ``fn`` on its tensors' device, with its ``stream`` argument as the
    current CUDA stream: its calls, and what they allocate, then belong to that
    stream."""
    @functools.wraps(fn)
    def wrapped(*args, stream=None, **kwargs):
        import torch
        km = _km()
        first = args[0] if args else kwargs.get("x", kwargs.get("dy"))
        km._on_gpu(first, "the first argument")
        with torch.cuda.device(first.device) if stream is None else torch.cuda.stream(km._stream_on(stream, first)):
            return fn(*args, **kwargs)
    return wrapped


def _km():
    import distance_argmin_gb300 as km
    return km


@_on_stream
def nearest_experts(x, centroids, ws=None):
    """Expert of each token: its nearest centroid -> int64 ids ``(n, 1)``.
    ``x`` (n, d) and ``centroids`` (n_experts, d) float32, n >= n_experts as
    kmeans_assign requires (fewer tokens: see ``few_nearest_experts``)."""
    labels, _, _ = _km().kmeans_assign(x, centroids, ws=ws)
    return labels.view(-1, 1)


@_on_stream
def few_nearest_experts(x, centroids):
    """nearest_experts for any number of tokens: fewer than the experts are
    repeated to as many rows as kmeans_assign wants."""
    n, k = x.shape[0], centroids.shape[0]
    if n >= k:
        return nearest_experts(x, centroids)
    padded = x.repeat((k + n - 1) // n, 1) if n else x.new_zeros(k, x.shape[1])
    return nearest_experts(padded, centroids)[:n]


class Saved:
    """What experts_forward keeps for experts_backward."""

    def __init__(self, **kept):
        self.__dict__.update(kept)


@_on_stream
def experts_forward(x, ids, w1, w2, b1=None, b2=None, weights=None, residual=None, activation="gelu", keep=False):
    """``(y, saved)``: y (n, d_out) of tokens x (n, d), float16 or bfloat16.

    ``ids`` (n, topk) experts of each token (negative: none); ``w1`` (n_experts,
    hidden, d), ``b1`` (n_experts, hidden), ``w2`` (n_experts, d_out, hidden),
    ``b2`` (n_experts, d_out); ``weights`` (n, topk) float32, ones by default;
    ``residual`` (n, d_out).  ``keep``: hold what the gradient needs in
    ``saved``, else None."""
    km = _km()
    n_experts = w1.shape[0]
    offsets, _, rows = km.kmeans_route(ids, n_experts)
    xs = km.kmeans_route_gather(x, rows, offsets)
    h, pre = km.kmeans_linear(xs, w1, bias=b1, offsets=offsets, activation=activation, save_pre=keep)
    ys, _ = km.kmeans_linear(h, w2, bias=b2, offsets=offsets)
    y = km.kmeans_route_combine(ys, rows, offsets, weights=weights, residual=residual)
    saved = Saved(offsets=offsets, rows=rows, xs=xs, pre=pre, h=h, ys=ys, weights=weights, activation=activation,
                  has_b1=b1 is not None, has_b2=b2 is not None) if keep else None
    return y, saved


@_on_stream
def experts_backward(dy, saved, w1, w2):
    """Gradients of experts_forward -> dict with ``x``, ``w1``, ``b1``, ``w2``,
    ``b2`` and ``weights`` (None where the forward pass had none); the
    residual's gradient is ``dy``."""
    km = _km()
    s = saved
    weights = s.weights
    if weights is None:
        import torch
        weights = torch.ones(s.rows.shape, dtype=torch.float32, device=dy.device)
    dys, dweights = km.kmeans_route_combine_grad(dy, s.ys, s.rows, s.offsets, weights)
    dh, dw2, db2 = km.kmeans_linear_grad(dys, s.h, w2, offsets=s.offsets, need_db=s.has_b2)
    dxs, dw1, db1 = km.kmeans_linear_grad(dh, s.xs, w1, pre=s.pre, offsets=s.offsets, activation=s.activation,
                                          need_db=s.has_b1)
    dx = km.kmeans_route_combine(dxs, s.rows, s.offsets)
    return {"x": dx, "w1": dw1, "b1": db1, "w2": dw2, "b2": db2,
            "weights": dweights if s.weights is not None else None}


@_on_stream
def block_forward(x, gate_w, w1, w2, topk, norm_weight=None, norm_bias=None, b1=None, b2=None, gate_bias=None,
                  scores="softmax", groups=1, topk_groups=None, renormalize=True, scale=1.0, eps=1e-5,
                  activation="gelu", keep=False):
    """``(y, saved)``: y (n, d) = x + the gated experts of the normalised tokens.

        h = kmeans_layernorm(x, norm_weight, norm_bias)
        ids, weights = kmeans_gate(h gate_w^T, topk, ..)     gate_w (n_experts, d)
        y = experts_forward(h, ids, w1, w2, .., weights, residual=x)

    x (n, d) float16 or bfloat16, the experts' matrices as for experts_forward
    with d_out = d (up to ``LINEAR_MAX_EXPERTS`` of them, fewer than the gate
    alone takes); ``gate_bias`` (n_experts,) float32 and the options from
    ``scores`` to ``scale`` are kmeans_gate's.  The router's logits are a
    kmeans_linear's, in x's 16-bit type: the gate orders the rounded ones.  ``keep``: hold what the gradient
    needs in ``saved``, else None."""
    km = _km()
    h, mean, rstd = km.kmeans_layernorm(x, norm_weight, norm_bias, eps=eps, save_stats=keep)
    logits, _ = km.kmeans_linear(h, gate_w)
    ids, weights = km.kmeans_gate(logits, topk, scores=scores, bias=gate_bias, groups=groups, topk_groups=topk_groups,
                                  renormalize=renormalize, scale=scale)
    y, saved = experts_forward(h, ids, w1, w2, b1, b2, weights=weights, residual=x, activation=activation, keep=keep)
    if keep:
        saved.__dict__.update(x=x, normed=h, mean=mean, rstd=rstd, logits=logits, ids=ids, how=dict(
            scores=scores, renormalize=renormalize, scale=scale), has_norm_weight=norm_weight is not None,
            has_norm_bias=norm_bias is not None)
    return y, saved


@_on_stream
def block_backward(dy, saved, gate_w, w1, w2, norm_weight=None):
    """Gradients of block_forward -> dict with ``x``, ``gate_w``, ``w1``, ``b1``,
    ``w2``, ``b2``, ``norm_weight`` and ``norm_bias`` (None where the forward
    pass had none).  ``norm_weight``: the forward pass's, if it had one."""
    km = _km()
    s = saved
    if (norm_weight is not None) != s.has_norm_weight:
        raise ValueError("norm_weight must be given where block_forward had one, and only there")
    dys, dweights = km.kmeans_route_combine_grad(dy, s.ys, s.rows, s.offsets, s.weights)
    dlogits = km.kmeans_gate_grad(dweights, s.logits, s.ids, **s.how)
    dh, dgate_w, _ = km.kmeans_linear_grad(dlogits, s.normed, gate_w, need_db=False)
    dhid, dw2, db2 = km.kmeans_linear_grad(dys, s.h, w2, offsets=s.offsets, need_db=s.has_b2)
    dxs, dw1, db1 = km.kmeans_linear_grad(dhid, s.xs, w1, pre=s.pre, offsets=s.offsets, activation=s.activation,
                                          need_db=s.has_b1)
    # the experts' way back to the tokens takes the gate's along
    dh = km.kmeans_route_combine(dxs, s.rows, s.offsets, residual=dh)
    dx, dnorm_weight, dnorm_bias = km.kmeans_layernorm_grad(dh, s.x, s.mean, s.rstd, weight=norm_weight, residual=dy,
                                                            need_dweight=s.has_norm_weight, need_dbias=s.has_norm_bias)
    return {"x": dx, "gate_w": dgate_w, "w1": dw1, "b1": db1, "w2": dw2, "b2": db2, "norm_weight": dnorm_weight,
            "norm_bias": dnorm_bias}

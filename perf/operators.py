"""Cases of the expert-routing and expert-product operators, for measurement.

Three operators, each with its directions:

* ``route``: slots (token, choice) sorted by expert, and the tokens' rows
  copied into that order;
* ``combine``: the experts' rows brought back to their tokens with weights
  and a residual ("fwd"), and its gradient ("bwd");
* ``linear``: rows times their expert's matrix with bias, activation and
  residual ("fwd"; ``pre`` also keeps the values before the activation), and
  its gradient ("bwd").  One expert without offsets is an ordinary dense
  layer.

``run`` computes a case either with elementary torch operations in float32
(``own`` false) or through the package's entry points (``own`` true).
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"float32": torch.float32, "float16": torch.float16, "bfloat16": torch.bfloat16}
ROOT_2_OVER_PI = math.sqrt(2.0 / math.pi)


def listed():
    return [
        # one token of a served request on its way to two experts
        dict(name="route_token", op="route", n=1, topk=2, experts=16, d=2048, dtype="bfloat16", drop=0.0),
        # a prefill's tokens, four choices each, some dropped by a capacity limit
        dict(name="route_prefill", op="route", n=8192, topk=4, experts=64, d=4096, dtype="bfloat16", drop=0.05),
        # samples sent to the cluster they were assigned to (65536 x 2048 float32, 1024 clusters)
        dict(name="route_clusters", op="route", n=65536, topk=1, experts=1024, d=2048, dtype="float32", drop=0.0),
        # a decode batch brought back to its tokens
        dict(name="combine_decode", op="combine", direction="fwd", n=16, topk=8, experts=64, d=4096, dtype="bfloat16",
             drop=0.0, residual=True),
        # odd sizes: rows that are not a multiple of 16 bytes, tokens with no kept choice among them
        dict(name="combine_odd", op="combine", direction="fwd", n=4097, topk=3, experts=24, d=1031, dtype="float16",
             drop=0.1, residual=True),
        # a training step's way back through the weighted sum
        dict(name="combine_train", op="combine", direction="bwd", n=16384, topk=8, experts=128, d=2048,
             dtype="bfloat16", drop=0.02, residual=False),
        # one token through a dense layer
        dict(name="linear_token", op="linear", direction="fwd", m=1, experts=1, active=1, dropped=0, n=8192, k=2048,
             dtype="bfloat16", activation="gelu", bias=True, residual=False, pre=False),
        # a decode batch whose rows went to 20 of 64 experts
        dict(name="linear_decode", op="linear", direction="fwd", m=24, experts=64, active=20, dropped=0, n=4096,
             k=2048, dtype="bfloat16", activation="silu", bias=True, residual=False, pre=False),
        # a dense layer over a long prefill, added to the residual stream
        dict(name="linear_dense", op="linear", direction="fwd", m=8192, experts=1, active=1, dropped=0, n=8192,
             k=2048, dtype="bfloat16", activation="gelu_tanh", bias=True, residual=True, pre=False),
        # a training step's forward over ragged groups, empty experts and dropped rows among them
        dict(name="linear_ragged", op="linear", direction="fwd", m=12347, experts=64, active=57, dropped=77, n=4096,
             k=2048, dtype="float16", activation="silu", bias=True, residual=False, pre=True),
        # the same layer's gradient on few large experts
        dict(name="grad_ragged", op="linear", direction="bwd", m=16384, experts=32, active=30, dropped=0, n=4096,
             k=2048, dtype="bfloat16", activation="gelu", bias=True, residual=False, pre=True),
        # the gradient of a small dense layer of odd row count and ragged widths
        dict(name="grad_small", op="linear", direction="bwd", m=257, experts=1, active=1, dropped=0, n=1000, k=520,
             dtype="float16", activation="relu", bias=True, residual=False, pre=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    v = _log_int(rng, lo, hi)
    return v if rng.random() < 0.3 else max(64, v // 64 * 64)


def draw(rng):
    op = rng.choice(["route", "combine", "linear", "linear"])
    dtype = rng.choice(["bfloat16", "bfloat16", "float16"])
    if op in ("route", "combine"):
        if rng.random() < 0.25:
            dtype = "float32"
        n = _log_int(rng, 1, 65536)
        experts = _log_int(rng, 2, 1024)
        topk = min(experts, rng.randint(1, 8))
        d = _width(rng, 64, 8192)
        d = max(1, min(d, (1 << 29) // (n * topk * (4 if dtype == "float32" else 2))))
        case = dict(op=op, n=n, topk=topk, experts=experts, d=d, dtype=dtype, drop=rng.choice([0.0, 0.0, 0.02, 0.2]))
        if op == "combine":
            case["direction"] = rng.choice(["fwd", "bwd"])
            case["residual"] = case["direction"] == "fwd" and rng.random() < 0.5
        return case
    direction = rng.choice(["fwd", "bwd"])
    m = _log_int(rng, 1, 16384)
    experts = 1 if rng.random() < 0.4 else _log_int(rng, 2, 64)
    active = min(m, experts, max(1, int(experts * rng.uniform(0.4, 1.0))))
    n = _width(rng, 64, 8192)
    k = _width(rng, 64, 4096)
    n = max(64, min(n, (1 << 29) // (experts * k), (1 << 36) // (max(m, 1) * k)))
    dropped = rng.randint(0, max(0, m - active) // 16) if experts > 1 else 0
    return dict(op="linear", direction=direction, m=m, experts=experts, active=active, dropped=dropped, n=n, k=k,
                dtype=dtype, activation=rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"]),
                bias=rng.random() < 0.7, residual=direction == "fwd" and rng.random() < 0.4,
                pre=direction == "bwd" or rng.random() < 0.4)


def _choices(case, g):
    """(n, topk) int64 experts, distinct per token, some popular, and -1 where a choice was dropped."""
    n, topk, experts = case["n"], case["topk"], case["experts"]
    bias = torch.randn(experts, generator=g, device="cuda")
    score = torch.rand(n, experts, generator=g, device="cuda").clamp_(1e-6, 1 - 1e-6)
    score = bias - torch.log(-torch.log(score))
    ids = torch.topk(score, topk, dim=1).indices if topk > 1 else score.argmax(dim=1, keepdim=True)
    lost = torch.rand(n, topk, generator=g, device="cuda") < case["drop"]
    return torch.where(lost, torch.full_like(ids, -1), ids)


def _counts(case, seed):
    """Rows of each expert: `active` of them have at least one, some many."""
    r = np.random.RandomState(seed % (2 ** 32))
    rows = case["m"] - case["dropped"]
    chosen = np.sort(r.permutation(case["experts"])[:case["active"]])
    share = np.exp(0.5 * r.randn(case["active"]))
    extra = r.multinomial(rows - case["active"], share / share.sum())
    counts = np.zeros(case["experts"], dtype=np.int64)
    counts[chosen] = 1 + extra
    return counts


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dt)

    if case["op"] == "route":
        return dict(case=case, experts=_choices(case, g), x=normal(case["n"], case["d"]))
    if case["op"] == "combine":
        n, topk, d = case["n"], case["topk"], case["d"]
        offsets, _, rows = _sorted_slots(_choices(case, g), case["experts"])
        weights = torch.softmax(torch.randn(n, topk, generator=g, device="cuda"), dim=1)
        s = dict(case=case, offsets=offsets, rows=rows, weights=weights, ys=normal(n * topk, d))
        if case["direction"] == "bwd":
            s["dy"] = normal(n, d)
        elif case["residual"]:
            s["residual"] = normal(n, d)
        return s
    m, n, k, experts = case["m"], case["n"], case["k"], case["experts"]
    counts = _counts(case, seed)
    shape = (experts, n, k) if experts > 1 else (n, k)
    s = dict(case=case, x=normal(m, k), w=normal(*shape, scale=k ** -0.5))
    if experts > 1:
        off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        s["offsets"] = torch.from_numpy(off).cuda()
        s["cap"] = int(counts.max())
    if case["direction"] == "bwd":
        s["dy"] = normal(m, n)
        s["pre"] = normal(m, n)
    else:
        if case["bias"]:
            s["bias"] = normal(*shape[:-1], scale=0.5)
        if case["residual"]:
            s["residual"] = normal(m, n)
    return s


# ------------------------------------------------------------- plain forms
def _sorted_slots(ids, experts):
    key = torch.where(ids.reshape(-1) < 0, experts, ids.reshape(-1))
    order = torch.argsort(key, stable=True)
    rows = torch.empty_like(order)
    rows[order] = torch.arange(order.numel(), device=order.device)
    edges = torch.arange(experts + 1, device=order.device)
    offsets = torch.searchsorted(key[order], edges)
    return offsets.int(), order.int(), rows.int().view(ids.shape)


def _activate(z, name):
    if name == "relu":
        return torch.clamp(z, min=0)
    if name == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(ROOT_2_OVER_PI * (z + 0.044715 * z * z * z)))
    if name == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _slope(z, name):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        t = torch.tanh(ROOT_2_OVER_PI * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * ROOT_2_OVER_PI * (1 + 3 * 0.044715 * z * z)
    if name == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    return torch.ones_like(z)


def _padded(s):
    """Row index (experts, cap) of every expert's rows, and which of them exist."""
    off = s["offsets"].long()
    at = off[:-1, None] + torch.arange(s["cap"], device=off.device)
    real = at < off[1:, None]
    return torch.where(real, at, 0), real


def _plain_linear(s):
    case, dt = s["case"], s["x"].dtype
    x, w = s["x"].float(), s["w"].float()
    if case["experts"] == 1:
        z = x @ w.t()
        if "bias" in s:
            z = z + s["bias"].float()
        y = _activate(z, case["activation"])
        if "residual" in s:
            y = y + s["residual"].float()
    else:
        at, real = _padded(s)
        zp = torch.bmm(x[at], w.transpose(1, 2))
        if "bias" in s:
            zp = zp + s["bias"].float()[:, None, :]
        z = torch.zeros(case["m"], case["n"], device=x.device)
        y = torch.zeros_like(z)
        rows = at[real]
        z[rows] = zp[real]
        yp = _activate(zp[real], case["activation"])
        if "residual" in s:
            yp = yp + s["residual"].float()[rows]
        y[rows] = yp
    return {"y": y.to(dt), "pre": z.to(dt)} if case["pre"] else {"y": y.to(dt)}


def _plain_linear_grad(s):
    case, dt = s["case"], s["x"].dtype
    x, w = s["x"].float(), s["w"].float()
    dz = s["dy"].float() * _slope(s["pre"].float(), case["activation"])
    if case["experts"] == 1:
        dx, dw, db = dz @ w, dz.t() @ x, dz.sum(0)
    else:
        at, real = _padded(s)
        dzp = dz[at] * real[:, :, None]
        dxp = torch.bmm(dzp, w)
        dx = torch.zeros_like(x)
        dx[at[real]] = dxp[real]
        dw, db = torch.bmm(dzp.transpose(1, 2), x[at]), dzp.sum(1)
    out = {"dx": dx.to(dt), "dw": dw.to(dt)}
    if case["bias"]:
        out["db"] = db.to(dt)
    return out


def _plain(s):
    case = s["case"]
    if case["op"] == "route":
        offsets, order, rows = _sorted_slots(s["experts"], case["experts"])
        kept = torch.arange(order.numel(), device=order.device) < offsets[-1]
        xs = s["x"][(order // case["topk"]).long()] * kept[:, None]
        return {"offsets": offsets, "order": order, "rows": rows, "xs": xs}
    if case["op"] == "combine":
        rows, weights = s["rows"].long(), s["weights"]
        kept = rows < s["offsets"][-1]
        dt = s["ys"].dtype
        back = torch.where(kept[:, :, None], s["ys"][rows].float(), 0.0)
        if case["direction"] == "fwd":
            y = (back * weights[:, :, None]).sum(1)
            if "residual" in s:
                y = y + s["residual"].float()
            return {"y": y.to(dt)}
        dy = s["dy"].float()
        dys = torch.empty(s["ys"].shape, device=dy.device)
        dys[rows.reshape(-1)] = ((weights * kept)[:, :, None] * dy[:, None, :]).reshape(-1, case["d"])
        return {"dys": dys.to(dt), "dweights": (back * dy[:, None, :]).sum(2)}
    return _plain_linear(s) if case["direction"] == "fwd" else _plain_linear_grad(s)


# ---------------------------------------------------- the package's operators
def _own(s):
    import distance_argmin_gb300 as km
    case = s["case"]
    if case["op"] == "route":
        if "ws" not in s:
            s["ws"] = km.route_workspace(case["n"], case["topk"], case["experts"])
        offsets, order, rows = km.kmeans_route(s["experts"], case["experts"], ws=s["ws"])
        xs = km.kmeans_route_gather(s["x"], rows, offsets)
        return {"offsets": offsets, "order": order, "rows": rows, "xs": xs}
    if case["op"] == "combine":
        if case["direction"] == "fwd":
            return {"y": km.kmeans_route_combine(s["ys"], s["rows"], s["offsets"], weights=s["weights"],
                                                 residual=s.get("residual"))}
        dys, dweights = km.kmeans_route_combine_grad(s["dy"], s["ys"], s["rows"], s["offsets"], s["weights"])
        return {"dys": dys, "dweights": dweights}
    if "ws" not in s:
        op = km.OP_LINEAR if case["direction"] == "fwd" else km.OP_LINEAR_GRAD
        s["ws"] = km.linear_workspace(op, case["m"], case["n"], case["k"], case["experts"])
    if case["direction"] == "fwd":
        y, pre = km.kmeans_linear(s["x"], s["w"], bias=s.get("bias"), residual=s.get("residual"),
                                  offsets=s.get("offsets"), activation=case["activation"], save_pre=case["pre"],
                                  ws=s["ws"])
        return {"y": y, "pre": pre} if case["pre"] else {"y": y}
    dx, dw, db = km.kmeans_linear_grad(s["dy"], s["x"], s["w"], pre=s["pre"], offsets=s.get("offsets"),
                                       activation=case["activation"], need_db=case["bias"], ws=s["ws"])
    return {"dx": dx, "dw": dw, "db": db} if case["bias"] else {"dx": dx, "dw": dw}


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    b = 4 if case["dtype"] == "float32" else 2
    if case["op"] == "route":
        n, slots, d = case["n"], case["n"] * case["topk"], case["d"]
        return {"bytes": slots * (8 + 4 + 4) + 4 * (case["experts"] + 1) + (n + slots) * d * b, "flops": 0}
    if case["op"] == "combine":
        n, slots, d = case["n"], case["n"] * case["topk"], case["d"]
        kept = slots * (1 - case["drop"])
        if case["direction"] == "fwd":
            return {"bytes": kept * d * b + n * d * b * (2 if case["residual"] else 1) + slots * 8,
                    "flops": 2 * kept * d}
        return {"bytes": (n + kept + slots) * d * b + slots * 12, "flops": 3 * kept * d}
    m, n, k, experts = case["m"], case["n"], case["k"], case["experts"]
    rows = m - case["dropped"]
    if case["direction"] == "fwd":
        values = rows * k + case["active"] * n * k + m * n * (1 + case["pre"]) + rows * n * case["residual"]
        return {"bytes": (values + case["active"] * n * case["bias"]) * b, "flops": 2 * rows * n * k}
    values = 2 * rows * n + rows * k + m * k + (case["active"] + experts) * n * k + experts * n * case["bias"]
    return {"bytes": values * b, "flops": 4 * rows * n * k}


# ------------------------------------------------------ definitions in 64 bits
def _phi(z):
    return 0.5 * torch.special.erfc(-z / math.sqrt(2.0))


def _f64(z, name):
    """The activation and its derivative in float64."""
    if name == "relu":
        return z.relu(), torch.where(z > 0, 1.0, 0.0).double()
    if name == "gelu":
        return z * _phi(z), _phi(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        u = math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
        du = math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z ** 2)
        sg = torch.sigmoid(2 * u)
        return z * sg, sg + 2 * z * sg * (1 - sg) * du
    if name == "silu":
        sg = torch.sigmoid(z)
        return z * sg, sg + z * sg * (1 - sg)
    return z, torch.ones_like(z)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "route":
        ids = s["experts"].reshape(-1).cpu().numpy()
        key = np.where(ids < 0, case["experts"], ids)
        order = np.lexsort((np.arange(key.size), key))
        kept = int((key < case["experts"]).sum())
        xs = torch.zeros(key.size, case["d"], dtype=torch.float64, device="cuda")
        xs[:kept] = s["x"].double()[torch.from_numpy(order[:kept] // case["topk"]).cuda()]
        return {"offsets": None, "order": None, "rows": None, "xs": xs}
    if case["op"] == "combine":
        last = int(s["offsets"][-1])
        w, ys = s["weights"].double(), s["ys"]
        if case["direction"] == "fwd":
            y = s["residual"].double() if "residual" in s else torch.zeros(case["n"], case["d"], dtype=torch.float64,
                                                                           device="cuda")
            for j in range(case["topk"]):
                r = s["rows"][:, j].long()
                t = (r < last).nonzero()[:, 0]
                y[t] += w[t, j, None] * ys[r[t]].double()
            return {"y": y}
        dy = s["dy"].double()
        dys = torch.zeros(ys.shape, dtype=torch.float64, device="cuda")
        dw = torch.zeros_like(w)
        for j in range(case["topk"]):
            r = s["rows"][:, j].long()
            t = (r < last).nonzero()[:, 0]
            dys[r[t]] = w[t, j, None] * dy[t]
            dw[t, j] = (dy[t] * ys[r[t]].double()).sum(1)
        return {"dys": dys, "dweights": dw}
    m, n, k = case["m"], case["n"], case["k"]
    if 4 * m * n * k > 1.2e12:
        return None
    edges = s["offsets"].tolist() if "offsets" in s else [0, m]
    w = s["w"].double().view(case["experts"], n, k)
    x = s["x"].double()
    if case["direction"] == "fwd":
        y = torch.zeros(m, n, dtype=torch.float64, device="cuda")
        z = torch.zeros_like(y)
        for e in range(case["experts"]):
            a, b = edges[e], edges[e + 1]
            z[a:b] = x[a:b] @ w[e].t()
            if "bias" in s:
                z[a:b] += s["bias"].double().view(case["experts"], n)[e]
            y[a:b] = _f64(z[a:b], case["activation"])[0]
            if "residual" in s:
                y[a:b] += s["residual"][a:b].double()
        return {"y": y, "pre": z} if case["pre"] else {"y": y}
    dz = s["dy"].double() * _f64(s["pre"].double(), case["activation"])[1]
    dx, dw = torch.zeros_like(x), torch.zeros_like(w)
    db = torch.zeros(case["experts"], n, dtype=torch.float64, device="cuda")
    for e in range(case["experts"]):
        a, b = edges[e], edges[e + 1]
        dx[a:b] = dz[a:b] @ w[e]
        dw[e] = dz[a:b].t() @ x[a:b]
        db[e] = dz[a:b].sum(0)
    out = {"dx": dx, "dw": dw.view(s["w"].shape)}
    if case["bias"]:
        out["db"] = db.view(s["w"].shape[:-1])
    return out

"""Cases for the layers of a model that answers from a table: layer norm, the choice of experts for
each row, the rows' way to their experts and back, and the softmax loss over a table's rows.

A case names the operator (``op``), its sizes and its type.  ``run`` computes it in elementary
torch operations, or, where ``own`` is true, through the package's entry points.

Sizes: 2048 and 16384 rows, 32768 pooled rows, tables of 100000 rows and the widths 128, 256, 512,
1024 and 4096 are those of the package's own workloads; the others are generic.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"fp32": 4, "fp16": 2, "bf16": 2}
EPS = 1e-5
PIECE = 1 << 27   # logits that the plain loss holds at a time


# ---------------------------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------------------------

def listed():
    return [
        # served users' states before the next layer: a small call, its latency counts
        dict(name="norm-2048x128-fp32", op="norm", rows=2048, cols=128, dtype="fp32", wide=False),
        # a training step at an odd width, rows of a wider buffer
        dict(name="norm-train-8191x1000-fp16", op="norm_train", rows=8191, cols=1000, dtype="fp16", wide=True),
        # a training step on the widest pooled batch
        dict(name="norm-train-32768x4096-bf16", op="norm_train", rows=32768, cols=4096, dtype="bf16", wide=False),
        # 64 requests choose 2 of 64 experts: the smallest call
        dict(name="route-64x64-fp32", op="route", rows=64, experts=64, k=2, scores="softmax", bias=False,
             groups=1, top_groups=1, renormalize=True, dtype="fp32"),
        # a training step with balanced sigmoid scores, 8 of 256 experts out of 4 of 8 groups
        dict(name="route-train-32768x256-bf16", op="route_train", rows=32768, experts=256, k=8, scores="sigmoid",
             bias=True, groups=8, top_groups=4, renormalize=True, dtype="bf16"),
        # the same 64 requests' rows go to their experts and come back
        dict(name="experts-64x512-bf16", op="experts", rows=64, experts=64, k=2, cols=512, left_out=0.0,
             dtype="bf16"),
        # a training step at an odd width, some choices dropped (full experts, padded rows)
        dict(name="experts-train-8191x250-fp32", op="experts_train", rows=8191, experts=13, k=3, cols=250,
             left_out=0.05, dtype="fp32"),
        # a training step of a large batch
        dict(name="experts-train-32768x1024-bf16", op="experts_train", rows=32768, experts=128, k=4, cols=1024,
             left_out=0.0, dtype="bf16"),
        # how likely the next events of 64 users were: the table is read once
        dict(name="loss-64x100000x128-bf16", op="loss", rows=64, vocab=100000, cols=128, dtype="bf16"),
        # a training step of a small odd table in full precision
        dict(name="loss-train-1000x9973x100-fp32", op="loss_train", rows=1000, vocab=9973, cols=100, dtype="fp32"),
        # a training step of one batch of users over one of the package's tables
        dict(name="loss-train-2048x100000x128-bf16", op="loss_train", rows=2048, vocab=100000, cols=128,
             dtype="bf16"),
        # a training step of a large batch over a wide table
        dict(name="loss-train-16384x131072x512-fp16", op="loss_train", rows=16384, vocab=131072, cols=512,
             dtype="fp16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A width on a log scale: a multiple of 64, of 8, or any number."""
    w = _log_int(rng, lo, hi)
    step = rng.choice((64, 64, 8, 1))
    return max(lo, min(hi, w // step * step))


def draw(rng):
    op = rng.choice(("norm", "norm_train", "route", "route_train", "experts", "experts_train", "loss",
                     "loss_train", "loss_train"))
    dtype = rng.choice(("bf16", "bf16", "fp16", "fp32"))
    if op in ("norm", "norm_train"):
        return dict(op=op, rows=_log_int(rng, 64, 32768), cols=_width(rng, 32, 4096), dtype=dtype,
                    wide=rng.random() < 0.3)
    if op in ("route", "route_train"):
        groups = rng.choice((1, 1, 2, 4, 8))
        experts = max(2, _log_int(rng, 8, 512) // groups) * groups
        top_groups = rng.randint(1, groups)
        return dict(op=op, rows=_log_int(rng, 1, 32768), experts=experts,
                    k=rng.randint(1, min(8, experts // groups * top_groups)),
                    scores=rng.choice(("softmax", "sigmoid")), bias=rng.random() < 0.5, groups=groups,
                    top_groups=top_groups, renormalize=rng.random() < 0.7, dtype=dtype)
    if op in ("experts", "experts_train"):
        cols, k = _width(rng, 32, 4096), rng.randint(1, 8)
        return dict(op=op, rows=_log_int(rng, 1, min(32768, (1 << 26) // (cols * k))),
                    experts=_log_int(rng, 2, 512), k=k, cols=cols, left_out=rng.choice((0.0, 0.0, 0.05, 0.3)),
                    dtype=dtype)
    cols = _width(rng, 32, 1024)
    rows = _log_int(rng, 1 if op == "loss" else 64, 16384)
    return dict(op=op, rows=rows, cols=cols, dtype=dtype,
                vocab=_log_int(rng, 500, max(1000, min(1 << 20, (1 << 37) // (rows * cols)))))


# ---------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------

def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    op, R = case["op"], case["rows"]

    def normal(*shape, scale=1.0, dtype=dt):
        v = torch.randn(*shape, generator=gen, device="cuda", dtype=dtype)
        return v if scale == 1.0 else v.mul_(scale)

    def uniform(*shape):
        return torch.rand(*shape, generator=gen, device="cuda")

    def integers(n, *shape):
        return torch.randint(n, shape, generator=gen, device="cuda")

    s = {"case": dict(case)}
    if op in ("norm", "norm_train"):
        C = case["cols"]
        wide = C + 24 if case["wide"] else C
        # rows with means and spreads of their own
        x = normal(R, wide, dtype=torch.float32) * (0.5 + uniform(R, 1)) + uniform(R, 1)
        s["x"] = x.to(dt)[:, :C]
        s["weight"] = normal(C, scale=0.1).add_(1)
        s["bias"] = normal(C, scale=0.1)
        if op == "norm_train":
            s["grad"] = normal(R, wide)[:, :C]
    elif op in ("route", "route_train"):
        E = case["experts"]
        # some experts are liked more than others, and the bias evens that out
        liked = normal(E, dtype=torch.float32)
        s["logits"] = (normal(R, E, dtype=torch.float32) + 0.5 * liked).to(dt)
        s["bias"] = liked.mul(-0.05) if case["bias"] else None
        if op == "route_train":
            s["grad"] = normal(R, case["k"], dtype=torch.float32)
    elif op in ("experts", "experts_train"):
        E, K, C = case["experts"], case["k"], case["cols"]
        # experts chosen more or less often, each at most once a row where there are enough
        liked = normal(1, E, dtype=torch.float32)
        ids = torch.argsort(uniform(R, E) + 0.2 * liked, dim=1)[:, :K].int()
        if E < K:
            ids = integers(E, R, K).int()
        s["ids"] = torch.where(uniform(R, K) < case["left_out"], -1, ids).int()
        w = uniform(R, K) + 0.1
        s.update(x=normal(R, C), y=normal(R * K, C), weights=w / w.sum(1, keepdim=True), residual=normal(R, C))
        if op == "experts_train":
            s.update(grad=normal(R, C), grad_rows=normal(R * K, C))
    else:
        V, C = case["vocab"], case["cols"]
        table = normal(V, C, scale=2 * C ** -0.5)
        # frequent and rare rows; some rows of the batch are padding
        targets = (V ** uniform(R)).long().sub_(1).clamp_(0, V - 1)
        s["x"] = (normal(R, C, dtype=torch.float32) + 1.5 * table[targets].float()).to(dt)
        s["targets"] = torch.where(uniform(R) < 0.05, -1, targets)
        s["table"] = table
        if op == "loss_train":
            # weighted rows, the mean's gradient; fp16 trains under a scale of the loss
            s["grad"] = (0.5 + uniform(R)) * ((65536.0 if case["dtype"] == "fp16" else 1.0) / R)
    return s


# ---------------------------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------------------------

def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    import table_embedding_bag_amd as tbe
    c = s["case"]
    op = c["op"]
    if op == "norm":
        y, _ = tbe.layer_norm(s["x"], s["weight"], s["bias"], eps=EPS, need_stats=False)
        return {"y": y}
    if op == "norm_train":
        y, stats = tbe.layer_norm(s["x"], s["weight"], s["bias"], eps=EPS)
        dx, dweight, dbias = tbe.layer_norm_backward(s["x"], stats, s["grad"], weight=s["weight"], bias=True)
        return {"y": y, "dx": dx, "dweight": dweight, "dbias": dbias}
    if op in ("route", "route_train"):
        ids, weights = tbe.route(s["logits"], c["k"], scores=c["scores"], bias=s["bias"], groups=c["groups"],
                                 top_groups=c["top_groups"], group_score=_group_score(c),
                                 renormalize=c["renormalize"])
        out = {"ids": ids, "weights": weights}
        if op == "route_train":
            out["dlogits"] = tbe.route_backward(s["logits"], ids, s["grad"], scores=c["scores"],
                                                renormalize=c["renormalize"])
        return out
    if op in ("experts", "experts_train"):
        plan = tbe.dispatch_plan(s["ids"], c["experts"])
        out = {"offsets": plan.offsets, "places": plan.places, "rows": tbe.dispatch(s["x"], plan),
               "y": tbe.combine(s["y"], plan, s["weights"], residual=s["residual"])}
        if op == "experts_train":
            dy, dweights = tbe.combine_backward(s["y"], plan, s["weights"], s["grad"])
            out.update(dy=dy, dweights=dweights, dx=tbe.dispatch_backward(s["grad_rows"], plan))
        return out
    loss, lse = tbe.softmax_loss(s["x"], s["table"], s["targets"])
    out = {"loss": loss, "lse": lse}
    if op == "loss_train":
        out["dx"], out["dtable"] = tbe.softmax_loss_backward(s["x"], s["table"], s["targets"], lse, s["grad"])
    return out


def _group_score(c):
    """Groups are chosen by their best two experts where there is a bias, else by the best."""
    return "top2" if c["bias"] and c["experts"] // c["groups"] > 1 else "max"


def _plain_norm(s):
    c = s["case"]
    dt = s["x"].dtype
    x = s["x"].float()
    mean = x.mean(1, keepdim=True)
    d = x - mean
    r = 1 / torch.sqrt((d * d).mean(1, keepdim=True) + EPS)
    n = d * r
    out = {"y": (n * s["weight"].float() + s["bias"].float()).to(dt)}
    if c["op"] == "norm_train":
        g = s["grad"].float()
        gw = g * s["weight"].float()
        dx = r * (gw - gw.mean(1, keepdim=True) - n * (gw * n).mean(1, keepdim=True))
        out.update(dx=dx.to(dt), dweight=(g * n).sum(0).to(dt), dbias=g.sum(0).to(dt))
    return out


def _plain_route(s):
    """In 64 bits: which experts are chosen hangs on scores next to each other."""
    c = s["case"]
    E, k, G = c["experts"], c["k"], c["groups"]
    x = s["logits"].double()
    R = x.shape[0]
    if c["scores"] == "softmax":
        e = torch.exp(x - x.amax(1, keepdim=True))
        p = e / e.sum(1, keepdim=True)
    else:
        p = 1 / (1 + torch.exp(-x))
    chosen_by = p if s["bias"] is None else p + s["bias"].double()
    if G > 1:
        best = torch.sort(chosen_by.view(R, G, E // G), dim=2, descending=True).values
        score = best[:, :, :2].sum(2) if _group_score(c) == "top2" else best[:, :, 0]
        top = torch.sort(score, dim=1, descending=True, stable=True).indices[:, :c["top_groups"]]
        inside = torch.zeros(R, G, dtype=torch.bool, device=x.device)
        inside[torch.arange(R, device=x.device)[:, None], top] = True
        chosen_by = torch.where(inside.repeat_interleave(E // G, dim=1), chosen_by, -math.inf)
    ids = torch.sort(chosen_by, dim=1, descending=True, stable=True).indices[:, :k]
    rows = torch.arange(R, device=x.device)[:, None]
    w = p[rows, ids]
    total = w.sum(1, keepdim=True)
    out = {"ids": ids.int(), "weights": (w / total if c["renormalize"] else w).float()}
    if c["op"] == "route_train":
        g = s["grad"].double()
        if c["renormalize"]:
            g = (g - (g * w).sum(1, keepdim=True) / total) / total
        dp = torch.zeros_like(p)
        dp[rows, ids] = g
        if c["scores"] == "softmax":
            dx = p * (dp - (p * dp).sum(1, keepdim=True))
        else:
            dx = dp * p * (1 - p)
        out["dlogits"] = dx.to(s["logits"].dtype)
    return out


def _plain_experts(s):
    c = s["case"]
    R, K, C, E = c["rows"], c["k"], c["cols"], c["experts"]
    dt, dev = s["x"].dtype, s["x"].device
    flat = s["ids"].view(-1).long()
    real = (flat >= 0) & (flat < E)
    key = torch.where(real, flat, E)
    order = torch.sort(key, stable=True).indices
    place = torch.empty_like(order)
    place[order] = torch.arange(R * K, device=dev)
    counts = (key[:, None] == torch.arange(E, device=dev)).sum(0)
    offsets = torch.cat([torch.zeros(1, dtype=torch.long, device=dev), torch.cumsum(counts, 0)])
    inside = (torch.arange(R * K, device=dev) < offsets[-1])[:, None]
    rows = torch.where(inside, s["x"][order // K], 0)
    at, on = place.view(R, K), real.view(R, K)
    y = s["residual"].float()
    for j in range(K):
        y = y + torch.where(on[:, j:j + 1], s["y"][at[:, j]].float() * s["weights"][:, j:j + 1], 0)
    out = {"offsets": offsets, "places": torch.where(on, at, -1).int(), "rows": rows, "y": y.to(dt)}
    if c["op"] == "experts_train":
        g = s["grad"].float()
        wide = g[order // K] * s["weights"].view(-1)[order][:, None]
        out["dy"] = torch.where(inside, wide, 0).to(dt)
        dw = [(g * s["y"][at[:, j]].float()).sum(1) for j in range(K)]
        out["dweights"] = torch.where(on, torch.stack(dw, 1), 0)
        dx = torch.zeros_like(g)
        for j in range(K):
            dx = dx + torch.where(on[:, j:j + 1], s["grad_rows"][at[:, j]].float(), 0)
        out["dx"] = dx.to(dt)
    return out


def _plain_loss(s):
    c = s["case"]
    R, V = c["rows"], c["vocab"]
    dt = s["x"].dtype
    x, w, t = s["x"].float(), s["table"].float(), s["targets"]
    train = c["op"] == "loss_train"
    loss, lse = torch.empty(R, device=x.device), torch.empty(R, device=x.device)
    dx, dw = torch.empty_like(x), torch.zeros_like(w)
    step = max(1, PIECE // V)
    for r in range(0, R, step):   # some rows' logits at a time
        xr, tr = x[r:r + step], t[r:r + step]
        z = xr @ w.t()
        top = z.amax(1, keepdim=True)
        on, at = tr >= 0, tr.clamp(min=0)[:, None]
        zt = z.gather(1, at)
        z = z.sub_(top).exp_()
        total = z.sum(1, keepdim=True)
        loss[r:r + step] = torch.where(on, (top - zt + torch.log(total))[:, 0], 0)
        lse[r:r + step] = (top + torch.log(total))[:, 0]
        if train:
            g = torch.where(on, s["grad"][r:r + step], 0)[:, None]
            z.div_(total)
            z.scatter_add_(1, at, torch.full_like(zt, -1.0))
            z.mul_(g)
            dx[r:r + step] = z @ w
            dw += z.t() @ xr
    out = {"loss": loss, "lse": lse}
    if train:
        out.update(dx=dx.to(dt), dtable=dw.to(dt))
    return out


def _run_plain(s):
    op = s["case"]["op"]
    if op in ("norm", "norm_train"):
        return _plain_norm(s)
    if op in ("route", "route_train"):
        return _plain_route(s)
    if op in ("experts", "experts_train"):
        return _plain_experts(s)
    return _plain_loss(s)


# ---------------------------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------------------------

def _exact_norm(s, train):
    x, w = s["x"].double(), s["weight"].double()
    var, mean = torch.var_mean(x, 1, correction=0, keepdim=True)
    sd = torch.sqrt(var + EPS)
    n = (x - mean) / sd
    out = {"y": n * w + s["bias"].double()}
    if train:
        g = s["grad"].double()
        a = g * w
        # the projection of a off the row's constant and off n
        C = x.shape[1]
        out["dx"] = (a - a.sum(1, keepdim=True) / C - n * ((a * n).sum(1, keepdim=True) / C)) / sd
        out["dweight"] = (g * n).sum(0)
        out["dbias"] = g.sum(0)
    return out


def _first_best(v):
    """The lowest index of each row's largest value."""
    n = v.shape[-1]
    at = torch.arange(n, device=v.device).expand_as(v)
    return torch.where(v == v.amax(-1, keepdim=True), at, n).amin(-1)


def _exact_route(s, train):
    c = s["case"]
    x = s["logits"].double()
    R, E = x.shape
    G, per = c["groups"], E // c["groups"]
    p = torch.softmax(x, 1) if c["scores"] == "softmax" else torch.sigmoid(x)
    by = p.clone() if s["bias"] is None else p + s["bias"].double()
    rows = torch.arange(R, device=x.device)
    if G > 1:
        left = by.view(R, G, per).clone()
        score = left.amax(2)
        if _group_score(c) == "top2":
            left.scatter_(2, _first_best(left)[:, :, None], -math.inf)
            score = score + left.amax(2)
        closed = torch.ones(R, G, dtype=torch.bool, device=x.device)
        for _ in range(c["top_groups"]):
            g = _first_best(score)
            closed[rows, g] = False
            score[rows, g] = -math.inf
        by.view(R, G, per)[closed] = -math.inf
    ids = []
    for _ in range(c["k"]):
        ids.append(_first_best(by))
        by[rows, ids[-1]] = -math.inf
    ids = torch.stack(ids, 1)
    w = p.gather(1, ids)
    q = w / w.sum(1, keepdim=True)
    out = {"ids": ids.int(), "weights": q if c["renormalize"] else w}
    if train:
        g = s["grad"].double()
        soft = c["scores"] == "softmax"
        if c["renormalize"]:
            # d log w of each chosen expert, and log w's slope in its logit
            d = q * (g - (q * g).sum(1, keepdim=True))
            d = d if soft else d * (1 - w)
            out["dlogits"] = torch.zeros_like(x).scatter_(1, ids, d)
        elif soft:
            out["dlogits"] = (-p * (w * g).sum(1, keepdim=True)).scatter_add_(1, ids, w * g)
        else:
            out["dlogits"] = torch.zeros_like(x).scatter_(1, ids, g * w * (1 - w))
    return out


def _exact_experts(s, train):
    c = s["case"]
    R, K, E = c["rows"], c["k"], c["experts"]
    ids = s["ids"].cpu().numpy().reshape(-1)
    lists = [np.flatnonzero(ids == e) for e in range(E)]          # assignments of each expert, in order
    sizes = [len(v) for v in lists]
    order = np.concatenate(lists)
    place = np.full(R * K, -1)
    place[order] = np.arange(len(order))
    dev = s["x"].device
    offsets = torch.from_numpy(np.concatenate([[0], np.cumsum(sizes)])).to(dev)
    at = torch.from_numpy(order).to(dev)
    token, n = at // K, len(order)
    out = {"offsets": offsets, "places": torch.from_numpy(place.reshape(R, K)).int().to(dev)}
    rows = torch.zeros(R * K, c["cols"], dtype=torch.float64, device=dev)
    rows[:n] = s["x"].double()[token]
    out["rows"] = rows
    w = s["weights"].double().reshape(-1)[at][:, None]
    out["y"] = s["residual"].double().index_add_(0, token, s["y"][:n].double() * w)
    if train:
        g = s["grad"].double()[token]
        dy = torch.zeros_like(rows)
        dy[:n] = g * w
        dw = torch.zeros(R * K, dtype=torch.float64, device=dev)
        dw[at] = (g * s["y"][:n].double()).sum(1)
        dx = torch.zeros(R, c["cols"], dtype=torch.float64, device=dev)
        out.update(dy=dy, dweights=dw.view(R, K), dx=dx.index_add_(0, token, s["grad_rows"][:n].double()))
    return out


def _exact_loss(s, train):
    x, w, t = s["x"].double(), s["table"].double(), s["targets"]
    R, V = x.shape[0], w.shape[0]
    loss, lse = (torch.zeros(R, dtype=torch.float64, device=x.device) for _ in range(2))
    dx, dw = torch.zeros_like(x), torch.zeros_like(w)
    for at in torch.arange(R, device=x.device).split(max(1, PIECE // 2 // V)):
        z = x[at] @ w.t()
        lse[at] = torch.logsumexp(z, 1)
        n = torch.nonzero(t[at] >= 0)[:, 0]     # the rows that have a target
        at, z = at[n], z[n]
        n = torch.arange(len(at), device=x.device)
        logp = torch.log_softmax(z, 1)
        loss[at] = -logp[n, t[at]]
        if train:
            d = logp.exp_()
            d[n, t[at]] -= 1
            d *= s["grad"][at].double()[:, None]
            dx[at] = d @ w
            dw.addmm_(d.t(), x[at])
    return {"loss": loss, "lse": lse, **({"dx": dx, "dtable": dw} if train else {})}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    train = op.endswith("_train")
    if op.startswith("norm"):
        return _exact_norm(s, train)
    if op.startswith("route"):
        return _exact_route(s, train)
    if op.startswith("experts"):
        return _exact_experts(s, train)
    return _exact_loss(s, train)


# ---------------------------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------------------------

def work(case):
    op, e, R = case["op"], BYTES[case["dtype"]], case["rows"]
    train = op.endswith("_train")
    if op.startswith("norm"):
        n, C = R * case["cols"], case["cols"]
        # forward: x, y; backward: x, dy, dx
        return {"bytes": n * e * (5 if train else 2) + C * e * (4 if train else 2),
                "flops": n * (18 if train else 8)}
    if op.startswith("route"):
        n, k = R * case["experts"], case["k"]
        return {"bytes": n * e * (3 if train else 1) + R * k * 8 + (R * k * 8 if train else 0)
                + (case["experts"] * 4 if case["bias"] else 0),
                "flops": n * (8 + k + (6 if train else 0))}
    if op.startswith("experts"):
        n, K = R * case["cols"], case["k"]
        kept = 1 - case["left_out"]
        # x to K rows; K rows and the residual to y; backwards y's gradient and K rows to K
        # rows' gradients; K rows' gradients to x's
        rows = (1 + K) + (K * kept + 2) + ((1 + K * kept + K) + (K * kept + 1) if train else 0)
        return {"bytes": int(n * e * rows) + R * K * (4 + 4 + 4 + (4 if train else 0)) + (case["experts"] + 1) * 8,
                "flops": int(n * K * (6 if train else 2))}
    V, C = case["vocab"], case["cols"]
    once = e * (R + V) * C
    return {"bytes": once * (2 if train else 1) + R * (16 + (8 if train else 0)),
            "flops": 2 * R * V * C * (3 if train else 1) + 4 * R * V}

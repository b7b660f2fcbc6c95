"""Cases for the layers that work on looked-up rows: the gated linear recurrence over jagged
sequences, the products grouped by ragged row ranges, and the counter-based dropout.

A case names the operator (``op``), its sizes and its type.  ``run`` computes it in elementary
torch operations, or, where ``own`` is true, through the package's entry points.

Sizes: 2048 bags of 1 to 32 lookups, 8192 bags of clip(Poisson(20), 0, 100) lookups, batches of
16384 and 32768 and the pooled widths 128, 256, 512, 1024 and 4096 are those of the
package's own workloads; the others are generic.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"fp32": 4, "fp16": 2, "bf16": 2}
ROUNDS = 7                       # Philox4x32 rounds of the dropout's generator
MUL = (0xD2511F53, 0xCD9E8D57)   # Philox4x32 multipliers (Salmon et al., SC'11)
WEYL = (0x9E3779B9, 0xBB67AE85)  # and key increments


# ---------------------------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------------------------

def listed():
    return [
        # one new event for each of 2048 served users: the smallest call, its latency counts
        dict(name="step-2048x128-fp32", op="step", seqs=2048, dim=128, dtype="fp32", gate="sigmoid"),
        # a training step on short histories, 1 to 32 events, odd width, x and the gate the two
        # halves of one projection (strided rows)
        dict(name="scan-2048-short-fp32", op="scan", seqs=2048, lengths="uniform", length=32,
             dim=100, dtype="fp32", gate="decay", halves=True),
        # a training step on medium histories, empty ones among them
        dict(name="scan-8192-medium-bf16", op="scan", seqs=8192, lengths="poisson", length=20,
             dim=256, dtype="bf16", gate="sigmoid", halves=False),
        # a training step on a few whole-life histories: long sequences, few rows
        dict(name="scan-4-long-bf16", op="scan", seqs=4, lengths="long", length=16384, dim=1024,
             dtype="bf16", gate="sigmoid", halves=True),
        # 64 requests spread over 64 experts: every weight is read for about one row
        dict(name="experts-serve-64-bf16", op="product", rows=64, groups=64, k=512, m=2048,
             dtype="bf16", sizes="random", bias=True),
        # a batch of pooled rows through one layer per domain, domains of very different sizes
        dict(name="experts-2048-fp16", op="product", rows=2048, groups=8, k=1024, m=512,
             dtype="fp16", sizes="skewed", bias=True),
        # a training step of a small odd layer in full precision
        dict(name="experts-train-odd-fp32", op="product_train", rows=8191, groups=5, k=250, m=130,
             dtype="fp32", sizes="random", bias=True),
        # a training step on a batch of pooled rows
        dict(name="experts-train-16384-bf16", op="product_train", rows=16384, groups=8, k=1024,
             m=4096, dtype="bf16", sizes="skewed", bias=True),
        # the same with more, larger experts
        dict(name="experts-train-32768-bf16", op="product_train", rows=32768, groups=16, k=4096,
             m=4096, dtype="bf16", sizes="random", bias=False),
        # dropout on one pooled table: a small call, its latency counts
        dict(name="dropout-2048x128-fp32", op="dropout", rows=2048, cols=128, dtype="fp32", p=0.1,
             residual=False, wide=False),
        # the gradient of dropout on an odd width, rows of a wider buffer
        dict(name="dropout-grad-8191x1000-fp16", op="dropout_grad", rows=8191, cols=1000,
             dtype="fp16", p=0.25, residual=False, wide=True),
        # dropout added to a residual, both directions, on the widest pooled batch
        dict(name="dropout-train-32768x4096-bf16", op="dropout_train", rows=32768, cols=4096,
             dtype="bf16", p=0.1, residual=True, wide=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A width on a log scale: a multiple of 64, of 8, or any number."""
    w = _log_int(rng, lo, hi)
    step = rng.choice((64, 64, 8, 1))
    return max(lo, min(hi, w // step * step))


def draw(rng):
    op = rng.choice(("step", "scan", "scan", "product", "product", "product_train", "dropout", "dropout_grad",
                     "dropout_train"))
    dtype = rng.choice(("bf16", "bf16", "fp16", "fp32"))
    if op == "step":
        return dict(op=op, seqs=_log_int(rng, 64, 32768), dim=_width(rng, 32, 1024), dtype=dtype,
                    gate=rng.choice(("sigmoid", "decay")))
    if op == "scan":
        lengths = rng.choice(("uniform", "poisson", "long"))
        length = {"uniform": _log_int(rng, 2, 512), "poisson": rng.randint(4, 60),
                  "long": _log_int(rng, 1024, 16384)}[lengths]
        dim = _width(rng, 32, 1024)
        most = max(1, min(8192, (1 << 26) // (length * dim)))   # tokens x width of at most 2^26
        return dict(op=op, seqs=_log_int(rng, max(1, most // 16), most), lengths=lengths,
                    length=length, dim=dim, dtype=dtype, gate=rng.choice(("sigmoid", "decay")),
                    halves=rng.random() < 0.5)
    if op in ("product", "product_train"):
        k, m = _width(rng, 64, 4096), _width(rng, 64, 4096)
        most = min(32768, (1 << 38) // (k * m))                 # at most half the largest listed one
        groups = _log_int(rng, 1, min(64, max(1, (1 << 28) // (k * m))))
        return dict(op=op, rows=_log_int(rng, 1 if op == "product" else 256, most), groups=groups, k=k, m=m, dtype=dtype,
                    sizes=rng.choice(("random", "skewed")), bias=rng.random() < 0.5)
    cols = _width(rng, 32, 4096)
    return dict(op=op, rows=_log_int(rng, 64, 32768), cols=cols, dtype=dtype,
                p=rng.choice((0.05, 0.1, 0.25, 0.5)),
                residual=op != "dropout_grad" and rng.random() < 0.5, wide=rng.random() < 0.3)


# ---------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------

def _lengths(case, g):
    """Lengths of the sequences: the same ones for every seed, in an order of its own."""
    S, L = case["seqs"], case["length"]
    fixed = np.random.default_rng([S, L])
    if case["lengths"] == "uniform":
        lengths = fixed.integers(1, L + 1, S)
    elif case["lengths"] == "poisson":
        lengths = np.clip(fixed.poisson(L, S), 0, 5 * L)
    else:
        lengths = fixed.integers(L - L // 8, L + 1, S)
    return g.permutation(lengths)


def _sizes(case, g):
    """Rows of each group: a uniform choice for each row, or one skewed as 1/rank with a group left empty."""
    G, N = case["groups"], case["rows"]
    p = np.full(G, 1.0 / G)
    if case["sizes"] == "skewed" and G > 1:
        p = 1.0 / np.arange(1, G + 1)
        g.shuffle(p)
        p[int(g.integers(G))] = 0.0
        p /= p.sum()
    return g.multinomial(N, p)


def _offsets(sizes):
    return torch.from_numpy(np.concatenate([[0], np.cumsum(sizes)]).astype(np.int64)).cuda()


def prepare(case, seed):
    host = np.random.default_rng([seed, 17])
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0):
        v = torch.randn(*shape, generator=gen, device="cuda", dtype=dt)
        return v if scale == 1.0 else v.mul_(scale)

    s = {"case": dict(case)}
    op = case["op"]
    if op in ("step", "scan"):
        S, D = case["seqs"], case["dim"]
        lengths = np.ones(S, dtype=np.int64) if op == "step" else _lengths(case, host)
        N = int(lengths.sum())
        if op == "scan" and case["halves"]:   # one projection gives both
            both = normal(N, 2 * D)
            x, gate = both[:, :D], both[:, D:]
        else:
            x, gate = normal(N, D), normal(N, D)
        # each channel remembers over a span of its own
        span = torch.rand(D, generator=gen, device="cuda") * 5
        if case["gate"] == "sigmoid":
            gate.add_(span.to(dt))
        else:
            gate.copy_(torch.sigmoid(gate.float() + span).to(dt))
        s.update(x=x, gate=gate, initial=torch.randn(S, D, generator=gen, device="cuda"))
        if op == "scan":
            s.update(offsets=_offsets(lengths), longest=int(lengths.max(initial=0)), grad_h=normal(N, D),
                     grad_final=torch.randn(S, D, generator=gen, device="cuda"))
    elif op in ("product", "product_train"):
        sizes = _sizes(case, host)
        G, N, K, M = case["groups"], case["rows"], case["k"], case["m"]
        s.update(x=normal(N, K), weight=normal(G, M, K, scale=K ** -0.5), offsets=_offsets(sizes),
                 ranges=np.concatenate([[0], np.cumsum(sizes)]).tolist(),
                 bias=normal(G, M, scale=0.1) if case["bias"] else None)
        if op == "product_train":
            s["grad"] = normal(N, M)
    else:
        R, C = case["rows"], case["cols"]
        wide = C + 24 if case["wide"] else C
        s.update(seed=int(host.integers(1 << 62)), offset=int(host.integers(1 << 40)))
        s["x"] = normal(R, wide)[:, :C]
        if op == "dropout_train":
            s["grad"] = normal(R, wide)[:, :C]
        s["residual"] = normal(R, C) if case["residual"] else None
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
    if op == "step":
        h, state = tbe.scan_step(s["x"], s["gate"], s["initial"], gate_kind=c["gate"])
        return {"h": h, "state": state}
    if op == "scan":
        h, final, carry = tbe.scan_forward(s["x"], s["gate"], s["offsets"], initial=s["initial"],
                                           gate_kind=c["gate"])
        dx, dgate, dinitial = tbe.scan_backward(s["x"], s["gate"], s["offsets"], carry, s["grad_h"],
                                                grad_final=s["grad_final"], initial=s["initial"],
                                                gate_kind=c["gate"])
        return {"h": h, "final": final, "dx": dx, "dgate": dgate, "dinitial": dinitial}
    if op == "product":
        return {"y": tbe.grouped_linear(s["x"], s["weight"], s["offsets"], bias=s["bias"])}
    if op == "product_train":
        y = tbe.grouped_linear(s["x"], s["weight"], s["offsets"], bias=s["bias"])
        dx, dw, db = tbe.grouped_linear_backward(s["x"], s["weight"], s["offsets"], s["grad"],
                                                 bias=s["bias"] is not None)
        return {"y": y, "dx": dx, "dw": dw, "db": db}
    if op == "dropout":
        return {"y": tbe.dropout(s["x"], c["p"], s["seed"], s["offset"], residual=s["residual"])}
    if op == "dropout_grad":
        return {"dx": tbe.dropout_backward(s["x"], c["p"], s["seed"], s["offset"])}
    y = tbe.dropout(s["x"], c["p"], s["seed"], s["offset"], residual=s["residual"])
    return {"y": y, "dx": tbe.dropout_backward(s["grad"], c["p"], s["seed"], s["offset"])}


def _doubling(a, b, place, longest):
    """v_i = a_i v_{i-1} + b_i within each sequence, spans doubled until the longest is covered;
    place: the index of each token within its sequence."""
    d = 1
    while d < longest:
        inside = (place[d:] >= d).unsqueeze(1)
        b, a = (torch.cat([b[:d], torch.where(inside, b[d:] + a[d:] * b[:-d], b[d:])]),
                torch.cat([a[:d], torch.where(inside, a[d:] * a[:-d], a[d:])]))
        d *= 2
    return b


def _gates(gate, kind):
    if kind == "decay":
        a = gate.float()
        return a, torch.ones_like(a)
    z = torch.exp(-gate.float().abs())
    hi, lo = 1 / (1 + z), z / (1 + z)
    up = gate >= 0
    return torch.where(up, hi, lo), torch.where(up, lo, hi)


def _plain_scan(s):
    c = s["case"]
    dt, off = s["x"].dtype, s["offsets"]
    N, S = s["x"].shape[0], c["seqs"]
    x = s["x"].float()
    a, b = _gates(s["gate"], c["gate"])
    lengths = off[1:] - off[:-1]
    seq = torch.repeat_interleave(torch.arange(S, device=x.device), lengths, output_size=N)
    place = torch.arange(N, device=x.device) - off[seq]
    left = lengths[seq] - 1 - place
    first, last, full = (place == 0).unsqueeze(1), (left == 0).unsqueeze(1), (lengths > 0).unsqueeze(1)
    initial, grad_final = s["initial"], s["grad_final"]
    h = _doubling(a, b * x + torch.where(first, a * initial[seq], 0), place, s["longest"])
    end = (off[1:] - 1).clamp(min=0)
    final = torch.where(full, h[end], initial)
    follow = torch.cat([a[1:], torch.zeros_like(a[:1])])      # a of the token after, 0 after a last one
    follow = torch.where(last, 0, follow)
    up = s["grad_h"].float() + torch.where(last, grad_final[seq], 0)
    lam = _doubling(follow.flip(0), up.flip(0), left.flip(0), s["longest"]).flip(0)
    before = torch.where(first, initial[seq], torch.cat([h[:1], h[:-1]]))
    dx = b * lam
    dgate = lam * before if c["gate"] == "decay" else lam * (before - x) * a * b
    at = off[:-1].clamp(max=max(N - 1, 0))
    dinitial = torch.where(full, a[at] * lam[at], grad_final)
    return {"h": h.to(dt), "final": final, "dx": dx.to(dt), "dgate": dgate.to(dt), "dinitial": dinitial}


def _plain_product(s, train):
    x, w, bias, r = s["x"], s["weight"], s["bias"], s["ranges"]
    G, M, K = w.shape
    y = torch.empty(x.shape[0], M, dtype=x.dtype, device=x.device)
    out = {"y": y}
    if train:
        out.update(dx=torch.empty_like(x), dw=torch.empty_like(w),
                   db=None if bias is None else torch.empty_like(bias))
    for g in range(G):   # one product for each group
        lo, hi = r[g], r[g + 1]
        wg, xg = w[g].float(), x[lo:hi].float()
        yg = xg @ wg.t()
        y[lo:hi] = yg if bias is None else yg + bias[g].float()
        if train:
            dy = s["grad"][lo:hi].float()
            out["dx"][lo:hi] = dy @ wg
            out["dw"][g] = dy.t() @ xg
            if bias is not None:
                out["db"][g] = dy.double().sum(0)
    return out


def _plain_words(blocks, first, seed, device):
    """Philox4x32 words of the counters first .. first + blocks - 1, [blocks, 4] in int64."""
    low = 0xFFFFFFFF
    n = torch.arange(blocks, device=device, dtype=torch.int64) + first
    v = [n & low, n >> 32, torch.zeros_like(n), torch.zeros_like(n)]
    key = [seed & low, seed >> 32]
    for _ in range(ROUNDS):
        hi, lo = [], []
        for m, w in ((MUL[0], v[0]), (MUL[1], v[2])):
            hi.append((w * (m >> 16) + (w * (m & 0xFFFF) >> 16)) >> 16)
            lo.append(w * m & low)
        v = [hi[1] ^ v[1] ^ key[0], lo[1], hi[0] ^ v[3] ^ key[1], lo[0]]
        key = [(k + w) & low for k, w in zip(key, WEYL)]
    return torch.stack(v, 1)


def _plain_dropout(x, residual, p, seed, offset):
    n = x.numel()
    words = _plain_words((n + 3) // 4, offset, seed, x.device)
    kept = (words >= int(p * 2.0 ** 32)).view(-1)[:n].view(x.shape)
    y = torch.where(kept, x.float() * (1 / (1 - p)), 0)
    if residual is not None:
        y = y + residual.float()
    return y.to(x.dtype)


def _run_plain(s):
    c = s["case"]
    op = c["op"]
    if op == "step":
        a, b = _gates(s["gate"], c["gate"])
        state = a * s["initial"] + b * s["x"].float()
        return {"h": state.to(s["x"].dtype), "state": state}
    if op == "scan":
        return _plain_scan(s)
    if op in ("product", "product_train"):
        return _plain_product(s, op == "product_train")
    if op == "dropout":
        return {"y": _plain_dropout(s["x"], s["residual"], c["p"], s["seed"], s["offset"])}
    if op == "dropout_grad":
        return {"dx": _plain_dropout(s["x"], None, c["p"], s["seed"], s["offset"])}
    y = _plain_dropout(s["x"], s["residual"], c["p"], s["seed"], s["offset"])
    return {"y": y, "dx": _plain_dropout(s["grad"], None, c["p"], s["seed"], s["offset"])}


# ---------------------------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------------------------

def _exact_scan(s, lengths):
    """One time step after another, on the sequences that are that long (longest first)."""
    c = s["case"]
    x, g = s["x"].double(), s["gate"].double()
    a, b = (torch.sigmoid(g), torch.sigmoid(-g)) if c["gate"] == "sigmoid" else (g, torch.ones_like(g))
    order = np.argsort(-lengths, kind="stable")
    start = torch.from_numpy((np.cumsum(lengths) - lengths)[order]).cuda()
    last = torch.from_numpy(lengths[order] - 1).cuda() + start
    back = torch.from_numpy(np.argsort(order)).cuda()
    sel = torch.from_numpy(order).cuda()
    active = [int((lengths > t).sum()) for t in range(int(lengths.max(initial=0)))]
    h, dx, dgate = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(x)
    before = torch.zeros_like(x)
    v = s["initial"].double()[sel]
    for t, n in enumerate(active):
        at = start[:n] + t
        before[at] = v[:n]
        v[:n] = a[at] * v[:n] + b[at] * x[at]
        h[at] = v[:n]
    final = v[back]
    up = s["grad_h"].double()
    mu = s["grad_final"].double()[sel]   # what the token after passes back
    for t, n in enumerate(active):
        at = last[:n] - t
        lam = up[at] + mu[:n]
        dx[at] = b[at] * lam
        dgate[at] = lam * (before[at] - x[at]) * a[at] * b[at] if c["gate"] == "sigmoid" else lam * before[at]
        mu[:n] = a[at] * lam
    return {"h": h, "final": final, "dx": dx, "dgate": dgate, "dinitial": mu[back]}


def _exact_kept(n, p, seed, offset):
    """Which of n elements are kept: Philox4x32 in numpy's unsigned 64-bit integers."""
    u = np.uint64
    low, sh = u(0xFFFFFFFF), u(32)
    ctr = np.arange((n + 3) // 4, dtype=np.uint64) + u(offset)
    c0, c1 = ctr & low, ctr >> sh
    c2, c3 = np.zeros_like(ctr), np.zeros_like(ctr)
    for r in range(ROUNDS):
        k0, k1 = u(((seed & 0xFFFFFFFF) + r * WEYL[0]) & 0xFFFFFFFF), u(((seed >> 32) + r * WEYL[1]) & 0xFFFFFFFF)
        p0, p1 = c0 * u(MUL[0]), c2 * u(MUL[1])
        c0, c1, c2, c3 = (p1 >> sh) ^ c1 ^ k0, p1 & low, (p0 >> sh) ^ c3 ^ k1, p0 & low
    least = math.floor(p * 2.0 ** 32)
    kept = np.empty((len(ctr), 4), dtype=bool)
    for i, w in enumerate((c0, c1, c2, c3)):
        kept[:, i] = w >= u(least)
    return torch.from_numpy(kept.reshape(-1)[:n]).cuda()


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "step":
        g, x, v = s["gate"].double(), s["x"].double(), s["initial"].double()
        v = torch.sigmoid(g) * v + torch.sigmoid(-g) * x if case["gate"] == "sigmoid" else g * v + x
        return {"h": v, "state": v}
    if op == "scan":
        return _exact_scan(s, _lengths(case, np.random.default_rng([seed, 17])))
    if op in ("product", "product_train"):
        sizes = s["offsets"].diff().tolist()
        xs = s["x"].double().split(sizes)
        w = s["weight"].double()
        y = [v @ w[g].t() for g, v in enumerate(xs)]
        if s["bias"] is not None:
            y = [v + s["bias"][g].double() for g, v in enumerate(y)]
        out = {"y": torch.cat(y)}
        if op == "product_train":
            dys = s["grad"].double().split(sizes)
            out["dx"] = torch.cat([v @ w[g] for g, v in enumerate(dys)])
            out["dw"] = torch.stack([v.t() @ u for v, u in zip(dys, xs)])
            out["db"] = None if s["bias"] is None else torch.stack([v.sum(0) for v in dys])
        return out
    n = case["rows"] * case["cols"]
    kept = _exact_kept(n, case["p"], s["seed"], s["offset"]).view(case["rows"], case["cols"])
    mapped = lambda v: torch.where(kept, v.double() / (1 - case["p"]), 0)  # noqa: E731
    y = mapped(s["x"])
    if op == "dropout_grad":
        return {"dx": y}
    if s["residual"] is not None:
        y = y + s["residual"].double()
    return {"y": y} if op == "dropout" else {"y": y, "dx": mapped(s["grad"])}


# ---------------------------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------------------------

def work(case):
    op, e = case["op"], BYTES[case["dtype"]]
    if op == "step":
        n = case["seqs"] * case["dim"]
        return {"bytes": n * (3 * e + 8), "flops": 8 * n}
    if op == "scan":
        n = int(_lengths(case, np.random.default_rng(0)).sum()) * case["dim"]
        states = case["seqs"] * case["dim"]
        # forward: x, gate, h; backward: x, gate, dh, dx, dgate; states: initial, final, and
        # initial, grad_final, dinitial
        return {"bytes": n * 8 * e + states * 4 * 5 + 16 * case["seqs"], "flops": 30 * n}
    if op in ("product", "product_train"):
        G, N, K, M = case["groups"], case["rows"], case["k"], case["m"]
        hit = G * (1 - (1 - 1 / G) ** N) if G > 1 else 1      # groups that hold a row
        bias = G * M * e if case["bias"] else 0
        fwd = {"bytes": e * (N * K + N * M + hit * K * M) + bias, "flops": 2 * N * K * M}
        if op == "product":
            return fwd
        return {"bytes": fwd["bytes"] + e * (2 * N * M + 2 * N * K + hit * K * M + G * K * M) + bias,
                "flops": 3 * fwd["flops"]}
    n = case["rows"] * case["cols"]
    streams = (3 if case["residual"] else 2) + (2 if op == "dropout_train" else 0)
    return {"bytes": n * e * streams, "flops": 2 * n}

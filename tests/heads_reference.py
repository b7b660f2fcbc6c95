"""Layer norm, the choice of experts, the rows' way to them and back, and the softmax loss from their
definitions in 64 bits, with bounds on what 32-bit arithmetic may be off by.

Every function takes torch tensors of float64 and returns {name: (value, bound)}: the bound before
the rounding to the output's type.  U32 is half a step of fp32, relative.
"""
import torch

U32 = 2.0 ** -24
TINY = {torch.float32: 2.0 ** -150, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def assert_close(got, ref, bound, what, dtype=None):
    """got within the bound of ref, and half a step of its own type."""
    dtype = dtype or got.dtype
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    if got.numel() == 0:
        return
    got = got.detach().double().to(ref.device)
    bound = bound + half_step(dtype) * (ref.abs() + bound) + TINY[dtype]
    bad = ~(((got - ref).abs() <= bound) | (got == ref) | (torch.isnan(got) & torch.isnan(ref)))
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {i}: got {got[i].item()!r}, "
                             f"expected {ref[i].item()!r} within {bound.expand_as(ref)[i].item()!r}")


# --- layer norm --------------------------------------------------------------------------------

def norm(x, w=None, b=None, eps=1e-5, g=None):
    """A row's sums in fp32: at most `chain` additions after each other."""
    N, D = x.shape
    chain = 48 + D / 1024
    ones = torch.ones(D, dtype=torch.float64, device=x.device)
    wt = ones if w is None else w
    m = x.mean(1, keepdim=True)
    d = x - m
    var = (d * d).mean(1, keepdim=True)
    r = 1 / torch.sqrt(var + eps)
    n = d * r
    y = n * wt + (0 if b is None else b)
    dm = (chain + 2) * U32 * x.abs().mean(1, keepdim=True)
    rel = (chain + 8) * U32 + dm * dm * r * r          # of r: half of the variance's, and its own
    dn = r * (dm + U32 * d.abs()) + n.abs() * (rel + U32)
    out = {"y": (y, wt.abs() * dn + 2 * U32 * (y.abs() + (n * wt).abs())),
           "mean": (m[:, 0], dm[:, 0]), "r": (r[:, 0], (rel * r)[:, 0])}
    if g is None:
        return out
    gw = g * wt
    s1, s2 = gw.mean(1, keepdim=True), (gw * n).mean(1, keepdim=True)
    dx = r * (gw - s1 - n * s2)
    e1 = (chain + 3) * U32 * gw.abs().mean(1, keepdim=True)
    e2 = (chain + 4) * U32 * (gw * n).abs().mean(1, keepdim=True) + (gw.abs() * dn).mean(1, keepdim=True)
    parts = gw.abs() + s1.abs() + (n * s2).abs()
    out["dx"] = (dx, r * (4 * U32 * parts + e1 + n.abs() * e2 + dn * s2.abs()) + rel * r * parts)
    # sums over rows: a workgroup's, then theirs
    chain = 128 + N / 512
    out["dweight"] = ((g * n).sum(0), chain * U32 * (g * n).abs().sum(0) + (g.abs() * dn).sum(0))
    out["dbias"] = (g.sum(0), chain * U32 * g.abs().sum(0))
    return out


# --- the choice of experts ---------------------------------------------------------------------

def _best(v):
    """The lowest index of each row's largest value."""
    at = torch.arange(v.shape[-1], device=v.device).expand_as(v)
    return torch.where(v == v.amax(-1, keepdim=True), at, v.shape[-1]).amin(-1)


def route(x, k, scores="softmax", bias=None, groups=1, top_groups=1, group_score="max", renormalize=True,
          scale=1.0, g=None):
    """ids (a tensor), weights, dlogits.  The choice without a bias is by the logits themselves."""
    x = torch.where(torch.isnan(x), -torch.inf, x.clamp(max=torch.finfo(torch.float32).max))
    N, E = x.shape
    top = x.amax(1, keepdim=True)
    top = torch.where(top == -torch.inf, 0, top)
    if scores == "softmax":
        e = torch.exp(x - top)
        z = e.sum(1, keepdim=True)
        p = torch.where(z > 0, e / z, 0)
    else:
        p = torch.sigmoid(x)
    summed = groups > 1 and group_score == "top2" and E // groups > 1
    by = (p + bias.double() if bias is not None else p.clone()) if bias is not None or summed else x.clone()
    rows = torch.arange(N, device=x.device)
    dead = torch.zeros(N, E, dtype=torch.bool, device=x.device)
    lowest = -torch.inf
    if groups > 1:
        left = by.reshape(N, groups, E // groups).clone()
        score = left.amax(2)
        if summed:
            left.scatter_(2, _best(left)[:, :, None], lowest)
            score = score + left.amax(2)
        closed = torch.ones(N, groups, dtype=torch.bool, device=x.device)
        for _ in range(top_groups):
            q = _first_of(score, ~closed)
            closed[rows, q] = False
        dead = closed.repeat_interleave(E // groups, dim=1)
    ids = []
    for _ in range(k):
        at = _first_of(by, dead)
        dead[rows, at] = True
        ids.append(at)
    ids = torch.stack(ids, 1)
    l = x.gather(1, ids)
    real = l > -torch.inf
    if scores == "softmax":
        lt = torch.where(real, l, -torch.inf).amax(1, keepdim=True)
        q = torch.where(real, torch.exp(l - torch.where(lt == -torch.inf, 0, lt)), 0)
    else:
        shift = l.amax(1, keepdim=True).clamp(max=0)
        shift = torch.where(shift == -torch.inf, 0, shift)
        q = torch.where(real, torch.exp(l.clamp(max=0) - shift) / (1 + torch.exp(-l.abs())), 0)
    total = q.sum(1, keepdim=True)
    q = torch.where(total > 0, q / total, 0)
    w = p.gather(1, ids)
    v = (q if renormalize else w) * scale
    # exponentials' arguments are rounded: relative errors of their size
    wide = torch.where(real, (l - top).abs().clamp(max=200) + l.abs().clamp(max=200), 0).amax(1, keepdim=True)
    rel = (2 * wide + 60) * U32
    out = {"ids": ids.int(), "weights": (v, rel * v.abs())}
    if g is not None:
        g = g * scale
        if renormalize:
            slope = 1 if scores == "softmax" else torch.sigmoid(-l)
            mean = torch.where(q > 0, q * g, 0).sum(1, keepdim=True)
            d = torch.where(q > 0, q * (g - mean), 0) * slope
            size = q * (g.abs() + (q * g).abs().sum(1, keepdim=True)) * slope
        else:
            slope = 1 if scores == "softmax" else torch.sigmoid(-l)
            d = torch.where(w > 0, w * g, 0) * slope
            size = d.abs()
        dx = torch.zeros_like(x).scatter_add_(1, ids, d)
        bound = torch.zeros_like(x).scatter_add_(1, ids, (rel + 20 * U32) * size)
        if scores == "softmax" and not renormalize:
            all_wide = (x - top).abs().clamp(max=200)
            dx = dx - p * d.sum(1, keepdim=True)
            bound = bound + ((2 * all_wide + 60) * U32 + rel) * p * d.abs().sum(1, keepdim=True) + 2.0 ** -148
        out["dlogits"] = (dx, bound)
    return out


def _first_of(v, dead):
    """The lowest index of each row's largest value that is not dead (infinities among them)."""
    at = torch.arange(v.shape[1], device=v.device).expand_as(v)
    top = torch.where(dead, -torch.inf, v).amax(1, keepdim=True)
    return torch.where((v == top) & ~dead, at, v.shape[1]).amin(1)


# --- rows to their experts and back ------------------------------------------------------------

def plan(ids, experts):
    flat = ids.reshape(-1).long().cpu()
    lists = [torch.nonzero(flat == e)[:, 0] for e in range(experts)]
    order = torch.cat(lists) if lists else torch.zeros(0, dtype=torch.long)
    places = torch.full((flat.numel(),), -1, dtype=torch.int32)
    places[order] = torch.arange(order.numel(), dtype=torch.int32)
    offsets = torch.tensor([0] + [len(v) for v in lists]).cumsum(0)
    return offsets, places.reshape(ids.shape)


def combine(y, places, weights=None, residual=None, g=None):
    N, k = places.shape
    on = (places >= 0)[:, :, None]
    rows = y[places.clamp(min=0).long()] if y.shape[0] else y.new_zeros(N, k, y.shape[1])
    rows = torch.where(on, rows, 0)
    w = torch.ones(N, k, dtype=torch.float64, device=y.device) if weights is None else weights
    w = torch.where(on[:, :, 0], w, 0)[:, :, None]
    out = (rows * w).sum(1) + (0 if residual is None else residual)
    size = (rows * w).abs().sum(1) + (0 if residual is None else residual.abs())
    res = {"out": (out, (k + 2) * U32 * size)}
    if g is not None:
        dy = torch.zeros_like(y)
        p = places[on[:, :, 0]].long()
        dy[p] = (g[:, None, :] * w)[on[:, :, 0]]
        res["dy"] = (dy, U32 * dy.abs())
        D = y.shape[1]
        res["dweights"] = ((g[:, None, :] * rows).sum(2), (D / 64 + 16) * U32 * (g[:, None, :] * rows).abs().sum(2))
    return res


# --- softmax loss ------------------------------------------------------------------------------

def loss(x, table, targets, scale=1.0, g=None, dtype=torch.float32):
    """dtype: of the rows, which the logits' gradients are rounded to."""
    N, D = x.shape
    V = table.shape[0]
    z = scale * x @ table.t()
    size = scale * x.abs() @ table.abs().t()
    dz = (D + 4) * U32 * size
    lse = torch.logsumexp(z, 1)
    p = torch.exp(z - lse[:, None])
    # the sum: its terms' errors, their exponents' (of values of that size), the additions'
    spread = (z - z.amax(1, keepdim=True)).abs() + z.abs().amax(1, keepdim=True)
    dlse = (p * (dz + 3 * U32 * spread)).sum(1) + (V / 64 + 256) * U32 + 3 * U32 * lse.abs()
    real = (targets >= 0) & (targets < V)
    at = torch.where(real, targets, 0).long()[:, None]
    zt = z.gather(1, at)[:, 0]
    value = torch.where(real, lse - zt, 0)
    out = {"lse": (lse, dlse), "loss": (value, torch.where(real, dlse + dz.gather(1, at)[:, 0] + 4 * U32 * zt.abs(), 0))}
    if g is not None:
        on = real[:, None]
        g = torch.where(real, g, 0)[:, None]
        d = p.clone()
        d[torch.arange(N, device=x.device), at[:, 0]] -= 1
        d = torch.where(on, d * g, 0)
        rel = dz + dlse[:, None] + 4 * U32 * (z.abs() + lse.abs()[:, None]) + 8 * U32
        # the machine's power of two gives 0 where it lies below the least normal number, 2^-126:
        # a probability, or |g| times it, is off by up to that much (fp16's factor takes more than
        # that off it again: it is 2^14 / max |g| at least)
        lost = 2.0 ** -126 * g.abs().clamp(min=1)
        dd = torch.where(on, g.abs() * p * rel + lost, 0) + 4 * U32 * d.abs()
        if dtype != torch.float32:
            dd = dd + half_step(dtype) * (d.abs() + dd)
        if dtype == torch.float16:   # 2^-25 of values that the largest row's 1 makes 2^14 at least
            dd = dd + 2.0 ** -39 * float(g.abs().max() if g.numel() else 0)
        x = torch.where(on, x, 0)
        out["dx"] = (scale * d @ table, scale * (dd @ table.abs() + (V + 16) * U32 * d.abs() @ table.abs()))
        out["dtable"] = (scale * d.t() @ x, scale * (dd.t() @ x.abs() + (N + 16) * U32 * d.abs().t() @ x.abs()))
    return out

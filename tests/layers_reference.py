"""The layers on looked-up rows from their definitions, in 64 bits on the CPU, with bounds on what
32-bit arithmetic may be off by (U32: half a step of fp32, relative)."""
import math

import numpy as np
import torch

U32 = 2.0 ** -24
MULTIPLIERS = (0xD2511F53, 0xCD9E8D57)
WEYL = (0x9E3779B9, 0xBB67AE85)
TINY = {torch.float32: 2.0 ** -150, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def rounded(bound, ref, dtype):
    """The bound of a value off by `bound` before its rounding to dtype."""
    return bound + half_step(dtype) * (np.abs(ref) + bound) + TINY[dtype]


def assert_close(got, ref, bound, what):
    got = got.detach().double().cpu().numpy()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    off = np.abs(got - ref)
    bad = ~((off <= bound) | (got == ref) | (np.isnan(got) & np.isnan(ref)))
    if bad.any():
        at = np.argwhere(bad)[0]
        i = tuple(at)
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} off, first at {i}: got {got[i]!r}, "
                             f"expected {ref[i]!r} within {np.broadcast_to(bound, ref.shape)[i]!r}")


# --- dropout -----------------------------------------------------------------------------------

def philox(counter, seed, rounds=7):
    """The four words of one Philox4x32 block, in Python integers."""
    c = [counter & 0xFFFFFFFF, counter >> 32 & 0xFFFFFFFF, 0, 0]
    k = [seed & 0xFFFFFFFF, seed >> 32]
    for _ in range(rounds):
        p0, p1 = c[0] * MULTIPLIERS[0], c[2] * MULTIPLIERS[1]
        c = [p1 >> 32 ^ c[1] ^ k[0], p1 & 0xFFFFFFFF, p0 >> 32 ^ c[3] ^ k[1], p0 & 0xFFFFFFFF]
        k = [(v + w) & 0xFFFFFFFF for v, w in zip(k, WEYL)]
    return c


def kept(n, p, seed, offset):
    least = math.floor(p * 2 ** 32)
    words = [w for b in range((n + 3) // 4) for w in philox((offset + b) % 2 ** 64, seed)]
    return np.array([w >= least for w in words[:n]], dtype=bool)


# --- gated linear recurrence -------------------------------------------------------------------

def gates(g, kind):
    if kind == "decay":
        return g, np.ones_like(g)
    z = np.exp(-np.abs(g))
    hi, lo = 1 / (1 + z), z / (1 + z)
    return np.where(g >= 0, hi, lo), np.where(g >= 0, lo, hi)


# What one step of a recurrence is off by, in U32 of its terms' magnitudes: a gate 5 (its
# exponential 2, the sum 1, the quotient 1, and the exponential once more in the sum), the product
# 1, the sum 1; 8 covers it.  A state that comes out of products of gates and partial sums over
# spans of tokens instead of one token after another takes no more than that for each of the
# tokens it passes.
STEP = 8


def scan(x, gate, offsets, initial, kind, grad_h=None, grad_final=None):
    """Every output and its bound before rounding: {name: (value, bound)}, all float64 arrays."""
    x, gate = x.astype(np.float64), gate.astype(np.float64)
    N, D = x.shape
    S = len(offsets) - 1
    a, b = gates(gate, kind)
    zero = np.zeros((S, D))
    initial = zero if initial is None else np.broadcast_to(initial, (S, D)).astype(np.float64)
    gh = np.zeros((N, D)) if grad_h is None else grad_h.astype(np.float64)
    gf = zero if grad_final is None else grad_final.astype(np.float64)
    u = STEP * U32
    new = lambda: np.zeros((N, D))  # noqa: E731
    h, eh, dx, edx, dg, edg = new(), new(), new(), new(), new(), new()
    before, big, ebefore = new(), new(), new()
    final, efinal, dinit, edinit = initial.copy(), zero.copy(), gf.copy(), zero.copy()
    with np.errstate(all="ignore"):
        for s in range(S):
            v, m, e = initial[s], np.abs(initial[s]), np.zeros(D)
            for t in range(offsets[s], offsets[s + 1]):
                before[t], big[t], ebefore[t] = v, m, e
                v = a[t] * v + b[t] * x[t]
                m = np.abs(a[t]) * m + np.abs(b[t] * x[t])
                e = np.abs(a[t]) * e + u * m
                h[t], eh[t] = v, e
            final[s], efinal[s] = v, e
            mu, m, e = gf[s], np.abs(gf[s]), np.zeros(D)
            for t in range(offsets[s + 1] - 1, offsets[s] - 1, -1):
                lam, m, e = gh[t] + mu, np.abs(gh[t]) + m, e
                e = e + U32 * m
                dx[t] = b[t] * lam
                edx[t] = np.abs(b[t]) * (e + u * m)
                if kind == "sigmoid":
                    ab, d, size = a[t] * b[t], before[t] - x[t], big[t] + np.abs(x[t])
                    ed = ebefore[t] + U32 * size
                else:
                    ab, d, size, ed = 1.0, before[t], big[t], ebefore[t]
                dg[t] = lam * d * ab
                edg[t] = ab * (e * (size + ed) + m * ed + m * size * 14 * U32)
                mu, m, e = a[t] * lam, np.abs(a[t]) * m, np.abs(a[t]) * (e + u * m)
            dinit[s], edinit[s] = mu, e
    return {"h": (h, eh), "final": (final, efinal), "dx": (dx, edx), "dgate": (dg, edg),
            "dinitial": (dinit, edinit)}


# --- grouped linear layer ----------------------------------------------------------------------

def grouped(x, weight, offsets, bias=None, grad=None):
    """{name: (value, bound before rounding)}: a sum of n products in fp32, in any order, is off by
    at most n U32 of the sum of the products' magnitudes (and U32 more for each of the last
    additions); products of 16-bit factors are exact."""
    x, w = x.astype(np.float64), weight.astype(np.float64)
    (N, K), (G, M, _) = x.shape, w.shape
    y, ey = np.zeros((N, M)), np.zeros((N, M))
    out = {"y": (y, ey)}
    if grad is not None:
        dy = grad.astype(np.float64)
        dx, edx, dw, edw = np.zeros((N, K)), np.zeros((N, K)), np.zeros((G, M, K)), np.zeros((G, M, K))
        db, edb = np.zeros((G, M)), np.zeros((G, M))
        out.update(dx=(dx, edx), dw=(dw, edw), db=(db, edb))
    for g in range(G):
        r = slice(offsets[g], offsets[g + 1])
        n = r.stop - r.start
        y[r] = x[r] @ w[g].T
        size = np.abs(x[r]) @ np.abs(w[g].T)
        if bias is not None:
            y[r] += bias[g].astype(np.float64)
            size = size + np.abs(bias[g])
        ey[r] = (K + 2) * U32 * size
        if grad is not None:
            dx[r], edx[r] = dy[r] @ w[g], (M + 2) * U32 * (np.abs(dy[r]) @ np.abs(w[g]))
            dw[g], edw[g] = dy[r].T @ x[r], (n + 2) * U32 * (np.abs(dy[r]).T @ np.abs(x[r]))
            db[g], edb[g] = dy[r].sum(0), (n + 2) * U32 * np.abs(dy[r]).sum(0)
    return out

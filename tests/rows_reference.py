"""The operators over 8-bit rows, the norm and the router's choice in numpy, in 64 bits, from their
definitions."""
import numpy as np
import torch

DT = {"fp16": torch.float16, "bf16": torch.bfloat16}
HALF_ULP = {"fp16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"fp16": 2.0 ** -25, "bf16": 2.0 ** -134}   # half the smallest subnormal
OVER = {"fp16": 65504.0 + 16, "bf16": (2 - 2.0 ** -7 + 2.0 ** -8) * 2.0 ** 127}   # the least that rounds to infinity


def f64(t):
    return t.detach().double().cpu().numpy()


def padded(k):
    return -(-k // 128) * 128


def random_rows(rows, k, seed, full=False):
    """Codes of every value in [-127, 127] (``full``: -128 too), zeros in the padding, and scales over
    several binades, zeros among them."""
    rng = np.random.default_rng(seed)
    q = np.zeros((rows, padded(k)), np.int8)
    q[:, :k] = rng.integers(-128 if full else -127, 128, (rows, k))
    s = (0.01 * np.exp(rng.uniform(-3, 1, rows))).astype(np.float32)
    if rows > 2:
        s[rng.random(rows) < 0.02] = 0
    return q, s


def product(x, xs, w, ws, n, gated, dtype):
    """What y has to be, and how far it may be from that.

    The sum is a whole number below 2^53.  Three roundings of fp32 (the sum, its product with either scale, the
    powers of two being exact): a relative 3 u (1 + u)^2 < 3.01 u, u = 2^-24.  silu(g) u passes the errors of g and u on
    with the magnitudes of its derivatives, |silu'| <= 1.1, and adds its own evaluation, (|g| + 8) 2^-23 of it.  y is
    rounded once."""
    h = (x.astype(np.float64) @ w.astype(np.float64).T) * xs.astype(np.float64)[:, None] * ws.astype(np.float64)
    err = 3.01 * 2.0 ** -24 * np.abs(h)
    want = h
    if gated:
        g, u, eg, eu = h[:, :n], h[:, n:], err[:, :n], err[:, n:]
        silu = g / (1 + np.exp(-np.clip(g, -700, 700)))
        want = silu * u
        err = 1.1 * eg * (np.abs(u) + eu) + np.abs(silu) * eu + (np.abs(g) + 8) * 2.0 ** -23 * np.abs(want)
    return want, err + HALF_ULP[dtype] * (np.abs(want) + err) + TINY[dtype]


def check_product(y, x, xs, w, ws, gated, dtype, what):
    n = w.shape[0] // (2 if gated else 1)
    want, tol = product(x, xs, w, ws, n, gated, dtype)
    y = f64(y)
    # round to nearest takes a value to infinity from half a step past the largest finite one on, and only from there
    with np.errstate(invalid="ignore"):
        over = np.isinf(y) & (y * want > 0) & (np.abs(want) + (tol - HALF_ULP[dtype] * np.abs(want)) >= OVER[dtype])
        bad = ~((np.abs(y - want) <= tol) | over | (y == want))  # (the same infinity has no distance)
    assert not bad.any(), (what, np.argwhere(bad)[:4].tolist(), y[bad][:4], want[bad][:4], int(bad.sum()))


def norm(h, weight, eps):
    """y of the norm and its relative error in fp32.  The squares' sum: each of up to k / 64 + 16 roundings a
    value goes through (a value's own square, the sums of its thread, of the wave, of the workgroup), half of
    that after the root; 2 u for h, mean, eps, root and quotient each, and the products."""
    k = h.shape[1]
    y = h / np.sqrt((h * h).mean(1, keepdims=True) + eps) * weight
    return y, (k / 64 + 16 + 24) * 2.0 ** -24


def check_rows(codes, scales, y, rel, k, what):
    """8-bit rows of values that are y up to the relative error ``rel``."""
    q, s, rel = f64(codes), f64(scales), rel + 2.0 ** -22
    top = np.abs(y).max(1)
    assert (np.abs(s - top / 127) <= rel * top / 127 + 2.0 ** -149).all(), what
    assert (q[:, k:] == 0).all() and (np.abs(q) <= 127).all(), what
    with np.errstate(divide="ignore", invalid="ignore"):
        exact = np.where(top[:, None] > 0, y * 127 / top[:, None], 0)
    # the code nearest to a quotient that is off by its own and the maximum's error
    bad = ~(np.abs(q[:, :k] - exact) <= 0.5 + 2 * rel * np.abs(exact))
    assert not bad.any(), (what, np.argwhere(bad)[:4].tolist(), q[:, :k][bad][:4], exact[bad][:4])


def choice(logits, top, score="softmax", bias=None, groups=1, top_groups=1, best=1, renormalise=True, factor=1.0):
    """(gates, ids) of each token, one token and one expert after another; and the relative error of a gate.

    Gates in fp32: exp of a difference of logits d has 2 |d| + 8 units of 2^-24, its sum over E experts E more, and
    as many again the renormalisation."""
    logits = np.asarray(logits, np.float64)
    tokens, experts = logits.shape
    each = experts // groups
    gates, ids, rel = np.zeros((tokens, top)), np.full((tokens, top), -1, np.int32), np.zeros((tokens, top))
    big = float(np.finfo(np.float32).max)
    for t in range(tokens):
        l = np.where(np.isnan(logits[t]), -np.inf, np.minimum(logits[t], big))
        live = [e for e in range(experts) if l[e] > -np.inf]
        if not live:
            continue
        m = max(l[e] for e in live)
        if score == "softmax":
            p = np.exp(l - m) / np.exp(l[live] - m).sum()
            d = m - l
        else:
            with np.errstate(over="ignore"):
                p = 1 / (1 + np.exp(-l))
            d = np.abs(l)
        rank = {}
        for e in live:
            b = 0.0 if bias is None else float(bias[e])
            if not np.isnan(b) and b > -np.inf:
                # without a bias in the order of the logits, which is that of p
                rank[e] = (l[e],) if bias is None else (p[e] + b,)
        if groups > 1:
            value = {}
            for g in range(groups):
                r = sorted((rank[e][0] if best == 1 or bias is not None else p[e] for e in rank if e // each == g), reverse=True)
                if r:
                    value[g] = sum(r[:best])
            kept = sorted(value, key=lambda g: (-value[g], g))[:top_groups]
            rank = {e: r for e, r in rank.items() if e // each in kept}
        chosen = sorted(rank, key=lambda e: (-rank[e][0], e))[:top]
        # a common factor, exp(-c), keeps the chosen p from vanishing together where they are renormalised
        low = l if score == "softmax" else np.minimum(l, 0)
        c = max((low[e] for e in chosen), default=0)
        q = {e: np.exp(low[e] - c) / (1 if score == "softmax" else 1 + np.exp(-abs(l[e]))) for e in chosen}
        total = sum(q.values())
        for j, e in enumerate(chosen):
            ids[t, j] = e
            gates[t, j] = factor * (q[e] / total if renormalise else p[e])
            rel[t, j] = (4 * min(d[e], 200.0) + 32 + 2 * experts + 2 * top) * 2.0 ** -24
    return gates, ids, rel

"""The scored router in 64 bits, token by token: choice, weights and gradient,
from the formulas of include/moe.h (moe_router)."""
import numpy as np

EPS32 = 2.0 ** -24                  # half a step of fp32


def scores(l, score):
    """Scores of one token's logits (float64), masked ones 0."""
    l = np.asarray(l, dtype=np.float64)
    live = l > -np.inf              # False for -inf and NaN
    s = np.zeros_like(l)
    if not live.any():
        return s, live
    with np.errstate(over="ignore", invalid="ignore"):
        if score == "sigmoid":
            s[live] = 1.0 / (1.0 + np.exp(-l[live]))
        else:
            m = l[live].max()
            s[live] = np.where(l[live] == m, 1.0, np.exp(l[live] - m))
            s /= s.sum()
    return s, live


def choose(l, k, score="softmax", n_groups=1, topk_groups=1, group_rank=2, balance=None):
    s, live = scores(l, score)
    E = len(s)
    if balance is None and (n_groups == 1 or group_rank == 1):
        c = np.asarray(l, dtype=np.float64).copy()
    else:
        c = s + (0.0 if balance is None else np.asarray(balance, dtype=np.float64))
    c[~live | np.isnan(c)] = -np.inf
    allowed = np.ones(E, dtype=bool)
    if n_groups > 1:
        ranks = []
        for g in c.reshape(n_groups, -1):
            best = sorted((v for v in g if v > -np.inf), reverse=True)[:group_rank]
            ranks.append(sum(best) if best else -np.inf)
        kept = sorted(range(n_groups), key=lambda g: (-ranks[g], g))[:topk_groups]
        allowed = np.isin(np.arange(E) // (E // n_groups), kept)
    order = sorted(np.nonzero(allowed)[0], key=lambda e: (-c[e], e))
    return np.array(order[:k], dtype=np.int64)


def chosen_scores(l, idx, score, renormalise):
    """Scores of the slots, and for renormalised weights their logarithm-free
    shares (exact where the scores underflow together)."""
    s, _ = scores(l, score)
    if not renormalise:
        return s[idx]
    lj = np.asarray(l, dtype=np.float64)[idx]
    live = lj > -np.inf
    if not live.any():
        return np.zeros(len(idx))
    with np.errstate(over="ignore", invalid="ignore"):
        ls = lj.copy()
        if score == "sigmoid":
            ls[live] = -np.logaddexp(0.0, -lj[live])
        m = ls[live].max()
        q = np.where(live, np.where(ls == m, 1.0, np.exp(ls - m)), 0.0)
    return q / q.sum()


def weights(l, idx, score="softmax", renormalise=True, scale=1.0):
    return scale * chosen_scores(l, idx, score, renormalise)


def backward(dw, l, idx, score="softmax", renormalise=True, scale=1.0):
    """dL/dl of one token, and a bound of its fp32 error for each expert in
    units of EPS32 times a condition number."""
    s, live = scores(l, score)
    q = chosen_scores(l, idx, score, renormalise)
    g = scale * np.where(live[idx], np.asarray(dw, dtype=np.float64), 0.0)
    out, mag = np.zeros(len(s)), np.zeros(len(s))
    inner, inner_mag = float((q * g).sum()), float(np.abs(q * g).sum())
    for j, e in enumerate(idx):
        if renormalise:
            h, hm = q[j] * (g[j] - inner), q[j] * (abs(g[j]) + inner_mag)
        else:
            h, hm = q[j] * g[j], abs(q[j] * g[j])
        f = 1.0
        if score == "sigmoid":
            with np.errstate(over="ignore"):
                f = 1.0 / (1.0 + np.exp(float(l[e]))) if live[e] else 0.0
        out[e] += h * f
        mag[e] += hm * f
    if score == "softmax" and not renormalise:
        out -= s * inner
        mag += s * inner_mag
    return out, mag


def span(l):
    """How far the live logits reach below the largest: exp's argument carries
    half a step of that, so scores carry as many half steps."""
    l = np.asarray(l, dtype=np.float64)
    l = l[np.isfinite(l)]
    return float(np.ptp(l)) + float(np.abs(l).max()) if l.size else 0.0


def half_steps(E, l):
    """Half steps of fp32 that a score may be off by, relative to itself: expf 4
    (its argument's rounding `span` more), twice (numerator and terms of the sum), the
    sum of E values in a tree of E/32 + 5 levels, quotient, scale, products 8."""
    return 16 + E / 32 + 5 + 2 * span(l)

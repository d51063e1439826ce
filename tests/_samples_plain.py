"""Plain forms of rotary positions and of drawing a token, in 64 bits or more (numpy, host)."""
import math

import numpy as np

U = 2.0 ** -24


def frequencies(rot, base=10000.0, scaling="plain", factor=1.0, original=0.0, low=0.0, high=0.0):
    """(radians per position of each pair, factor on what is turned)."""
    i = np.arange(rot // 2)
    if scaling == "ntk" and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    f = base ** (-2.0 * i / rot)
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "bands":
        t = np.clip((original * f / (2 * math.pi) - low) / (high - low), 0, 1)
        return (1 - t) * f / factor + t * f, 1.0
    if scaling == "yarn":
        def at(r):
            return rot * math.log(original / (2 * math.pi * r)) / (2 * math.log(base))
        first, last = max(0.0, math.floor(at(high))), min(rot - 1.0, math.ceil(at(low)))
        t = np.clip((i - first) / (max(last, first + 0.001) - first), 0, 1)
        return t * f / factor + (1 - t) * f, 0.1 * math.log(factor) + 1.0
    return f, 1.0


def turn(x, pos, freq, scale, interleaved):
    """x [n][heads][D] at positions pos [n] -> (out, tol) in 64 bits.

    tol bounds the fp32 arithmetic: the angle is rounded to fp32 as at most one half turn (pi u), sine and cosine
    are good to 2 ulp (2 u each, their values being at most 1), the factor and the two products and the sum
    round once each (u of at most |a| + |b|, times the factor): (pi + 2 + 1 + 2) u < 9 u of |a| + |b|."""
    n, heads, D = x.shape
    rot = 2 * len(freq)
    two_pi = 8 * np.arctan(np.longdouble(1))
    angle = np.fmod(np.asarray(pos, np.longdouble)[:, None] * np.asarray(freq, np.float64).astype(np.longdouble), two_pi)
    c, s = np.cos(angle).astype(np.float64)[:, None], np.sin(angle).astype(np.float64)[:, None]
    y, tol = x.astype(np.float64).copy(), np.zeros(x.shape)
    a = slice(0, rot, 2) if interleaved else slice(0, rot // 2)
    b = slice(1, rot, 2) if interleaved else slice(rot // 2, rot)
    p, q = y[..., a].copy(), y[..., b].copy()
    y[..., a], y[..., b] = (p * c - q * s) * scale, (p * s + q * c) * scale
    tol[..., a] = tol[..., b] = 9 * U * abs(scale) * (np.abs(p) + np.abs(q))
    return y, tol


# A weight is off by at most 8 u of itself (the exponent is held in two floats, whose second adds under 2^-44 of it; ex2.approx is
# good to 2^-22 = 4 u, the factor for the second float and the product round once each, u; twice that u for what the second
# float's own terms round) and by half a unit of 2^-44; a sum of weights by as much.
WEIGHT = 8 * U
UNIT = 2.0 ** -45


def order(l):
    """Tokens by larger logit first, lower index among equals (-0 equals 0)."""
    return np.lexsort((np.arange(len(l)), -l))


def check_row(l, u, T, k, p, low, token, prob, probs):
    """Whether a drawn token (and its probability, and all of them) is what the settings say, up to WEIGHT and UNIT."""
    l = np.where(np.isnan(l), -np.inf, l.astype(np.float64)) + 0.0
    V = len(l)
    if T == 0:
        T, k = 1.0, 1
    m = l.max()
    with np.errstate(invalid="ignore"):
        w = np.where(l == m, 1.0, np.exp((l - m) / T))
    at = order(l)
    ranked = w[at]
    if 0 < k < V:
        ranked[k:] = 0
    total, before = ranked.sum(), np.concatenate([[0.0], np.cumsum(ranked)[:-1]])
    slack = 2 * WEIGHT * total + V * UNIT
    rank = np.empty(V, np.int64)
    rank[at] = np.arange(V)
    in_k = np.ones(V, bool) if not 0 < k < V else rank < k
    sure = may = in_k
    if p < 1:
        sure = sure & (before[rank] < p * total - slack)
        may = may & (before[rank] < p * total + slack)
        sure[at[0]] = True
    if low > 0 and m < np.inf:
        keep = l - m >= T * math.log(low)
        sure, may = sure & keep, may & keep
    live = w > UNIT
    assert may[token] and live[token], f"token {token} is not among the kept"
    if probs is not None:
        kept = probs > 0
        assert not np.any(kept & ~may), "a token that is filtered out has a probability"
        assert not np.any(sure & ~kept & (w > 1e-17)), "a kept token has no probability"
        w = np.where(kept, w, 0.0)
        W = w.sum()
        assert np.all(np.abs(probs - w / W) <= (2 * WEIGHT + 4 * U) * w / W + 2 * V * UNIT / W)
        assert probs[token] == prob
        slack = 2 * WEIGHT * W + V * UNIT
    else:
        w = np.where(may, w, 0.0)
        W = w.sum()
        edge = np.where(may & ~sure, w, 0.0).sum()  # the tokens at a border, which may be kept or not
        slack = 2 * WEIGHT * W + V * UNIT + edge
        assert abs(prob - w[token] / W) <= (2 * WEIGHT + 4 * U + 2 * edge / W) * prob + 2 * V * UNIT / W
    run = np.cumsum(w)
    assert run[token] > u * W - slack and run[token] - w[token] <= u * W + slack, "another token stands at u"

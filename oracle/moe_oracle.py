"""CPU oracle of the RMSNorm, router, expert-sorting, dispatch and combine
operators and their gradients, in float64 (test infrastructure; numpy alone).

Error bounds: standard forward error analysis with the unit roundoff u = 2^-24
of fp32 (a sum whose longest chain has d additions is off by at most d u
sum|terms|), first-order terms times 1.05 for the rest, plus half a step of the
result's type (``round_half``).
"""
from __future__ import annotations

import numpy as np

from .ffn_oracle import round_half
from .mx_oracle import FP32_U

MORE = 1.05


# --------------------------------------------------------------------------
# RMSNorm
# --------------------------------------------------------------------------

def rmsnorm(z, gamma, eps=1e-5):
    """(y, rsigma) of the rows of z, float64."""
    z = np.asarray(z, np.float64)
    with np.errstate(invalid="ignore", over="ignore"):
        rs = 1.0 / np.sqrt((z * z).mean(axis=1) + eps)
        return z * rs[:, None] * gamma, rs


def rmsnorm_rho(depth):
    """|rsigma - exact| <= rho rsigma: the squares (1) and their sum (depth), the division
    (1) and the addition of eps (1) under a root that halves them, the root and the
    reciprocal (1 each)."""
    return MORE * (0.5 * (depth + 3) + 2) * FP32_U


def rmsnorm_bound(y, depth, t):
    """Bound on |y - exact|: rsigma's error and two products, rounded to ``t``."""
    e = (rmsnorm_rho(depth) + 2 * FP32_U) * np.abs(y)
    return MORE * e + round_half(np.abs(y) + e, t)


def rmsnorm_backward(dy, z, gamma, rs, dz=None):
    """(dx, dgamma), float64."""
    xh = z * rs[:, None]
    g = dy * gamma
    dx = rs[:, None] * (g - xh * (g * xh).mean(axis=1, keepdims=True))
    return (dx if dz is None else dx + dz), (dy * xh).sum(axis=0)


def rmsnorm_backward_bounds(dy, z, gamma, rs, dz, depth, row_depth, t, tp):
    """Bounds on (|dx - exact|, |dgamma - exact|).  The mean: g and xh (1 each), their
    product, depth additions, 1 / H and the product with it (3).  dx: at most ten
    roundings of each of its three terms on the way to the last one."""
    u = FP32_U
    xh = np.abs(z * rs[:, None])
    g = np.abs(dy * gamma)
    terms = (g * xh).mean(axis=1, keepdims=True)
    r = rs[:, None]
    first = r * g + r * xh * terms + (0.0 if dz is None else np.abs(dz))
    e = MORE * ((depth + 6) * u * r * xh * terms + 10 * u * first)
    dx, dga = rmsnorm_backward(dy, z, gamma, rs, dz)
    ega = MORE * (row_depth + 3) * u * (np.abs(dy) * xh).sum(axis=0)
    return e + round_half(np.abs(dx) + e, t), ega + round_half(np.abs(dga) + ega, tp)


# --------------------------------------------------------------------------
# router
# --------------------------------------------------------------------------

def route_index(logits, k, bias=None):
    """The k largest of fl32(logit + bias) of each row, in falling order, ties to the lowest
    index, NaN last."""
    key = np.asarray(logits, np.float32)
    if bias is not None:
        with np.errstate(invalid="ignore"):
            key = (key + np.asarray(bias, np.float32)).astype(np.float32)
    nan = np.isnan(key)
    rank = np.where(nan, -np.inf, key.astype(np.float64))
    # last key first: NaN after all numbers, then falling values; lexsort is stable in the index
    order = np.stack([np.lexsort((-rank[r], nan[r])) for r in range(key.shape[0])])
    return order[:, :k].astype(np.int32)


def scores(logits, scoring):
    x = np.asarray(logits, np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        if scoring == "sigmoid":
            e = np.exp(-np.abs(x))
            return np.where(x >= 0, 1 / (1 + e), e / (1 + e))
        m = x.max(axis=1, keepdims=True)
        p = np.where(x == -np.inf, 0.0, np.exp(x - np.where(m == -np.inf, 0.0, m)))
        s = p.sum(axis=1, keepdims=True)
        return np.where(s == 0, 0.0, p / np.where(s == 0, 1.0, s))


def chosen_shares(logits, index, scoring):
    """The chosen experts' shares of the sum of their scores, which are taken relative to
    e^top (top the largest of the chosen logits, of logistic scores where it is negative):
    the factor cancels, and no sum underflows.  0 for an index outside the experts, and where
    all chosen logits are -inf."""
    x = np.asarray(logits, np.float64)
    live = (index >= 0) & (index < x.shape[1])
    v = np.where(live, np.take_along_axis(x, np.where(live, index, 0).astype(np.int64), axis=1), -np.inf)
    top = v.max(axis=1, keepdims=True)
    top = np.where(top == -np.inf, 0.0, np.minimum(top, 0.0) if scoring == "sigmoid" else top)
    with np.errstate(over="ignore", invalid="ignore"):
        p = np.exp(v - top) if scoring == "softmax" else 1 / (np.exp(top) + np.exp(top - v))
    p = np.where(v == -np.inf, 0.0, p)
    s = p.sum(axis=1, keepdims=True)
    return np.where(s == 0, 0.0, p / np.where(s == 0, 1.0, s))


def route_weights(logits, index, scoring, renormalise, scale):
    if renormalise:
        return scale * chosen_shares(logits, index, scoring)
    return scale * np.take_along_axis(scores(logits, scoring), index.astype(np.int64), axis=1)


def score_error(logits, scoring):
    """Relative error of a score in fp32, per row: the difference in the exponent (its
    rounding times its size), two units of the exponential (a unit is 2 u), a sum of at
    most 1024 terms in chains of 37, a division or a product with a reciprocal (3); the
    renormalisation has the same once more."""
    x = np.asarray(logits, np.float64)
    spread = np.abs(np.where(np.isfinite(x), x, 0.0)).max(axis=1, keepdims=True) * 2
    a = np.minimum(spread, 104.0) if scoring == "softmax" else 0.0 * spread
    return MORE * FP32_U * 2 * (a + 4 + 37 + 3 + 5)


def weight_error(logits, index, scoring, renormalise):
    """Relative error of a weight, per row: that of a score; shares of logistic scores have a
    difference in the exponent too (its rounding times its size) where the chosen logits are
    all negative."""
    e = score_error(logits, scoring)
    if scoring == "sigmoid" and renormalise:
        x = np.asarray(logits, np.float64)
        live = (index >= 0) & (index < x.shape[1])
        v = np.take_along_axis(x, np.where(live, index, 0).astype(np.int64), axis=1)
        top = np.where(live, v, -np.inf).max(axis=1, keepdims=True)
        low = np.where(live & np.isfinite(v), v, np.inf).min(axis=1, keepdims=True)
        spread = np.where(np.isfinite(top) & np.isfinite(low) & (top < 0), top - low, 0.0)
        e = e + MORE * FP32_U * 2 * np.minimum(spread, 104.0)
    return e


def route_weights_bound(logits, index, scoring, renormalise, scale):
    w = np.abs(route_weights(logits, index, scoring, renormalise, scale))
    return w * weight_error(logits, index, scoring, renormalise) + 2.0 ** -125 * abs(scale)


def route_backward(dweight, logits, index, scoring, renormalise, scale):
    """dlogits, by the chain rule through the scores.  An index outside the experts is a choice
    that was never made: the others' shares are of their sum alone."""
    x = np.asarray(logits, np.float64)
    T, E = x.shape
    p = scores(x, scoring)
    live = (index >= 0) & (index < E)
    at = np.where(live, index, 0).astype(np.int64)
    g = np.where(live, np.asarray(dweight, np.float64) * scale, 0.0)
    d = np.zeros((T, E))
    if renormalise:
        # of w_i = c_i / s with c_i' = c_i (logistic: times 1 - c_i): w_i (g_i - sum w g) c_i' / c_i
        w = chosen_shares(x, index, scoring)
        g = np.where(live, w * (g - (w * g).sum(axis=1, keepdims=True)), 0.0)
    for j in range(index.shape[1]):
        d[np.arange(T)[live[:, j]], at[live[:, j], j]] += g[live[:, j], j]
    if scoring == "sigmoid":
        return d * scores(-x, "sigmoid") * (1.0 if renormalise else p)
    return d if renormalise else p * (d - (d * p).sum(axis=1, keepdims=True))


def route_backward_bound(dweight, logits, index, scoring, renormalise, scale, t):
    """Each gradient is a score (or weight) times a difference of terms that are at most
    max|g| and sum w |g|: their errors relative to those, and twenty roundings."""
    x = np.asarray(logits, np.float64)
    E = x.shape[1]
    p = scores(x, scoring)
    live = (index >= 0) & (index < E)
    at = np.where(live, index, 0).astype(np.int64)
    c = np.where(live, np.take_along_axis(p, at, axis=1), 0.0)
    g = np.abs(np.where(live, np.asarray(dweight, np.float64) * scale, 0.0))
    w = chosen_shares(x, index, scoring) if renormalise else c
    size = np.zeros(x.shape)
    for j in range(index.shape[1]):
        size[np.arange(len(x))[live[:, j]], at[live[:, j], j]] += w[live[:, j], j] * g[live[:, j], j]
    both = (w * g).sum(axis=1, keepdims=True)
    of = np.zeros(x.shape)                                   # the factor of the sum: w of the chosen, p of all
    if renormalise:
        for j in range(index.shape[1]):
            of[np.arange(len(x))[live[:, j]], at[live[:, j], j]] = w[live[:, j], j]
    elif scoring == "softmax":
        of = p
    e = (size + of * both) * (3 * weight_error(x, index, scoring, renormalise) + 20 * FP32_U) + 2.0 ** -125 * (1 + g.max(axis=1, keepdims=True))
    d = route_backward(dweight, logits, index, scoring, renormalise, scale)
    return e + round_half(np.abs(d) + e, t)


# --------------------------------------------------------------------------
# slots sorted by expert, dispatch and combine
# --------------------------------------------------------------------------

def moe_sort(index, experts):
    """(group_m, row, slot): a stable sort of the slots by expert; slots of other indices have no row."""
    flat = np.asarray(index).reshape(-1)
    live = (flat >= 0) & (flat < experts)
    order = np.argsort(np.where(live, flat, experts), kind="stable")
    kept = int(live.sum())
    slot = np.full(flat.size, -1, np.int32)
    slot[:kept] = order[:kept]
    row = np.full(flat.size, -1, np.int32)
    row[order[:kept]] = np.arange(kept)
    return np.bincount(flat[live], minlength=experts).astype(np.int32), row.reshape(np.shape(index)), slot


def moe_combine(y, row, weight=None, residual=None):
    """(out, sum of the terms' magnitudes), float64."""
    T, k = row.shape
    out = np.zeros((T, y.shape[1])) if residual is None else np.array(residual, np.float64)
    size = np.abs(out)
    for j in range(k):
        live = row[:, j] >= 0
        v = y[row[live, j]] * (1.0 if weight is None else weight[live, j, None])
        out[live] += v
        size[live] += np.abs(v)
    return out, size


def moe_combine_bound(out, size, k, t):
    e = MORE * (k + 1) * FP32_U * size
    return e + round_half(np.abs(out) + e, t)


def moe_dweight(dout, y, row):
    """(dweight, sum of the terms' magnitudes), float64."""
    T, k = row.shape
    d, size = np.zeros((T, k)), np.zeros((T, k))
    for j in range(k):
        live = row[:, j] >= 0
        v = dout[live] * y[row[live, j]]
        d[live, j], size[live, j] = v.sum(axis=1), np.abs(v).sum(axis=1)
    return d, size


def moe_dweight_bound(size, hidden):
    """A lane's chain has at most hidden / 32 + 8 products, the warp's sum five additions."""
    return MORE * (hidden // 32 + 16) * FP32_U * size + 2.0 ** -149

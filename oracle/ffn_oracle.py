"""CPU oracle of the LayerNorm and gated feed-forward operators, forward and
backward, in float64 (test infrastructure; numpy alone).

Sources of the definitions: te.LayerNorm as the drop-in of torch.nn.LayerNorm
(leeroopedia "FP8 Training Quickstart"), its epsilon 1e-5 (TE "Getting
Started", JAX page) and the fused LayerNormMLP on both pages; MXFP8 as in
``mx_oracle``.  The gated feed-forward replaces the MLP's first Linear by two
of the same input, h = act(x W_gate^T) * (x W_up^T).

Error bounds: standard forward error analysis with the unit roundoff u = 2^-24
of fp32 (a sum whose longest chain has d additions is off by at most d u
sum|terms|), first-order terms times 1.05 for the rest, plus half a step of the
result's type (``round_half``).
"""
from __future__ import annotations

import numpy as np

from .mx_oracle import FP32_U

HALF_STEP = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}     # relative, at most
# half the distance between the type's smallest subnormals (2^-133, 2^-24, 2^-149)
HALF_SUBNORMAL = {"bf16": 2.0 ** -134, "fp16": 2.0 ** -25, "fp32": 2.0 ** -150}


def round_half(v, t: str):
    """Largest error of rounding values up to |v| to the type ``t``."""
    return HALF_STEP[t] * np.abs(v) + HALF_SUBNORMAL[t]


# --------------------------------------------------------------------------
# LayerNorm
# --------------------------------------------------------------------------

def layernorm(x, gamma, beta=None, eps=1e-5):
    """(y, mu, rsigma) of the rows of x, float64."""
    x = np.asarray(x, np.float64)
    with np.errstate(invalid="ignore", over="ignore"):
        mu = x.mean(axis=1)
        d = x - mu[:, None]
        rs = 1.0 / np.sqrt((d * d).mean(axis=1) + eps)
        y = d * rs[:, None] * gamma
    return (y if beta is None else y + beta), mu, rs


def layernorm_stat_bounds(x, eps, depth):
    """|mu - exact| <= dmu, |rsigma - exact| <= rho rsigma for sums of longest chain ``depth``."""
    u, mu = FP32_U, x.mean(axis=1)
    var = ((x - mu[:, None]) ** 2).mean(axis=1)
    dmu = (depth + 1) * u * np.abs(x).mean(axis=1)
    rho = 0.5 * ((depth + 5) * u + (dmu ** 2 + 2 * u * np.abs(mu) * dmu) / (var + eps)) + 2 * u
    return 1.05 * dmu, 1.05 * rho


def layernorm_bound(x, gamma, beta, eps, depth, t):
    """Bound on |y - exact|: fp32 evaluation of fl(fl(x - mu) rs) gamma + beta, rounded to ``t``."""
    u = FP32_U
    y, mu, rs = layernorm(x, gamma, beta, eps)
    dmu, rho = layernorm_stat_bounds(x, eps, depth)
    xh = np.abs(x - mu[:, None]) * rs[:, None]
    e = 1.05 * (np.abs(gamma) * (rs[:, None] * dmu[:, None] + xh * (rho[:, None] + 3 * u)) + u * np.abs(y))
    return e + round_half(np.abs(y) + e, t)


def layernorm_backward(dy, x, gamma, mu, rs):
    """(dx, dgamma, dbeta) from the saved statistics, float64."""
    xh = (x - mu[:, None]) * rs[:, None]
    g = dy * gamma
    c1, c2 = g.mean(axis=1), (g * xh).mean(axis=1)
    dx = rs[:, None] * (g - c1[:, None] - xh * c2[:, None])
    return dx, (dy * xh).sum(axis=0), dy.sum(axis=0)


def layernorm_backward_bounds(dy, x, gamma, mu, rs, depth, row_depth, t, tp):
    """Bounds on dx, dgamma, dbeta for row sums of longest chain ``depth`` and
    column sums of longest chain ``row_depth`` (types ``t`` and ``tp``)."""
    u = FP32_U
    # xh: one rounding of x - mu and one of the product (or one of an fma whose
    # constant term mu rs is rounded on its own: |mu| rs u more)
    r = rs[:, None]
    xh = (x - mu[:, None]) * r
    exh = u * (2 * np.abs(xh) + 2 * np.abs(mu[:, None]) * r)
    g = dy * gamma
    c1, c2 = g.mean(axis=1)[:, None], (g * xh).mean(axis=1)[:, None]
    ec1 = (depth + 2) * u * np.abs(g).mean(axis=1)[:, None]
    ec2 = ((depth + 4) * u * np.abs(g * xh).mean(axis=1) + (np.abs(g) * exh).mean(axis=1))[:, None]
    e = r * (4 * u * (np.abs(g) + np.abs(c1) + np.abs(xh * c2)) + ec1 + np.abs(xh) * ec2 + np.abs(c2) * exh)
    dx, dga, dbe = layernorm_backward(dy, x, gamma, mu, rs)
    e = 1.05 * (e + u * np.abs(dx))
    ega = 1.05 * ((row_depth + 2) * u * np.abs(dy * xh).sum(axis=0) + (np.abs(dy) * exh).sum(axis=0))
    ebe = 1.05 * row_depth * u * np.abs(dy).sum(axis=0)
    return (e + round_half(np.abs(dx) + e, t), ega + round_half(np.abs(dga) + ega, tp),
            ebe + round_half(np.abs(dbe) + ebe, tp))


# --------------------------------------------------------------------------
# Gated feed-forward
# --------------------------------------------------------------------------

def sigmoid(x):
    x = np.asarray(x, np.float64)
    with np.errstate(over="ignore"):
        return np.where(x >= 0, 1.0 / (1.0 + np.exp(-np.abs(x))), np.exp(-np.abs(x)) / (1.0 + np.exp(-np.abs(x))))


_A = 2.0 * np.sqrt(2.0 / np.pi)


def act(x, kind):
    x = np.asarray(x, np.float64)
    if kind == "relu":
        return np.maximum(x, 0.0)
    if kind == "silu":
        return x * sigmoid(x)
    # (1 + tanh(z / 2)) / 2 is the logistic function of z, without the cancellation for x < 0
    return x * sigmoid(_A * (x + 0.044715 * x ** 3))


def act_grad(x, kind):
    x = np.asarray(x, np.float64)
    if kind == "relu":
        return (x > 0).astype(np.float64)
    if kind == "silu":
        s = sigmoid(x)
        return s + x * s * sigmoid(-x)
    z = _A * (x + 0.044715 * x ** 3)
    s = sigmoid(z)
    return s + x * s * sigmoid(-z) * _A * (1.0 + 3 * 0.044715 * x * x)


ACT_SLOPE = 1.13            # |act'| is below this for all three (gelu: 1.129)


def act_eval_error(x, kind):
    """Relative error of the fp32 activation x / (1 + 2^t) (and, with the same
    terms once more, of its derivative): t is off by a few u |t|, the hardware
    exponential and reciprocal by 2 ulp and 1 ulp."""
    x = np.abs(np.asarray(x, np.float64))
    t = np.zeros_like(x) if kind == "relu" else \
        np.minimum(1.4427 * (x if kind == "silu" else _A * (x + 0.044715 * x ** 3)), 200.0)
    return FP32_U * (16 + 4 * t)


def gated(g, u, kind):
    return act(g, kind) * u


def gated_bound(g, u, eg, eu, kind):
    """Bound on |h - act(g) u| in bf16 when the fp32 g and u are off by eg and eu."""
    a = np.abs(act(g, kind))
    ea = ACT_SLOPE * eg + (a + ACT_SLOPE * eg) * act_eval_error(g, kind) + 1e-36
    h = a * np.abs(u)
    e = 1.05 * (ea * (np.abs(u) + eu) + a * eu + 2 * FP32_U * h)
    return e + round_half(h + e, "bf16")


def gated_backward(dh, g, u, kind):
    """(dg, du), float64."""
    return dh * u * act_grad(g, kind), dh * act(g, kind)


def gated_backward_bounds(dh, g, u, kind):
    """Bounds on |dg| and |du| errors (fp32 evaluation, rounded to bf16).  The
    derivative is a sum of two terms, each off by act_eval_error relative to
    its own size (|x sigmoid'| <= 0.3 for silu, with the slope's factor below
    0.9 for gelu, where the terms can cancel)."""
    r = act_eval_error(g, kind)
    dg, du = gated_backward(dh, g, u, kind)
    if kind == "relu":
        terms = np.abs(act_grad(g, kind))
    else:
        z = g if kind == "silu" else _A * (g + 0.044715 * g ** 3)
        s = sigmoid(z)
        slope = 1.0 if kind == "silu" else _A * (1.0 + 3 * 0.044715 * g * g)
        terms = s + np.abs(g) * s * sigmoid(-z) * slope
    eg = 1.05 * np.abs(dh * u) * (2 * r * terms + 4 * FP32_U * terms + 1e-36)
    eu = 1.05 * np.abs(dh) * (np.abs(act(g, kind)) * (r + 2 * FP32_U) + 1e-36)
    return eg + round_half(np.abs(dg) + eg, "bf16"), eu + round_half(np.abs(du) + eu, "bf16")

"""The LayerNorm and gated feed-forward oracle against differences and
identities (CPU): every gradient equals the central difference of the forward
function, to the differences' own accuracy."""
import numpy as np
import pytest

from oracle import ffn_oracle as F
from oracle.mx_oracle import gelu_tanh

H = 1e-5            # step: central differences are off by ~ H^2 f''' / 6 and 2^-53 |f| / H


def difference(f, x, v):
    return (f(x + H * v) - f(x - H * v)) / (2 * H)


@pytest.mark.parametrize("rows,hidden", [(1, 1), (1, 2), (3, 7), (5, 64), (17, 100)])
def test_layernorm_gradients_are_the_differences(rows, hidden):
    rng = np.random.default_rng(rows * 100 + hidden)
    x = rng.standard_normal((rows, hidden)) * 2 + 0.5
    ga, be, dy = 1 + 0.1 * rng.standard_normal(hidden), rng.standard_normal(hidden), rng.standard_normal((rows, hidden))
    _, mu, rs = F.layernorm(x, ga, be)
    dx, dga, dbe = F.layernorm_backward(dy, x, ga, mu, rs)
    loss = lambda x, ga, be: (dy * F.layernorm(x, ga, be)[0]).sum()  # noqa: E731
    for seed in range(3):
        r = np.random.default_rng(seed)
        vx, vg = r.standard_normal(x.shape), r.standard_normal(hidden)
        scale = 1e-6 * (1 + np.abs(dy).sum())
        assert abs(difference(lambda t: loss(t, ga, be), x, vx) - (dx * vx).sum()) < scale
        assert abs(difference(lambda t: loss(x, t, be), ga, vg) - (dga * vg).sum()) < scale
        assert abs(difference(lambda t: loss(x, ga, t), be, vg) - (dbe * vg).sum()) < scale


@pytest.mark.parametrize("kind", ["silu", "gelu", "relu"])
def test_gated_gradients_are_the_differences(kind):
    rng = np.random.default_rng(3)
    g, u, dh = rng.standard_normal(400) * 3, rng.standard_normal(400), rng.standard_normal(400)
    g = np.where(np.abs(g) < 1e-3, 1e-3, g)                # (relu has no derivative at 0)
    dg, du = F.gated_backward(dh, g, u, kind)
    one = np.ones_like(g)
    assert np.allclose(dg, dh * difference(lambda t: F.gated(t, u, kind), g, one), atol=1e-8, rtol=1e-7)
    assert np.allclose(du, dh * difference(lambda t: F.gated(g, t, kind), u, one), atol=1e-8, rtol=1e-7)
    assert np.abs(F.act_grad(np.linspace(-30, 30, 200001), kind)).max() < F.ACT_SLOPE


def test_activations_at_their_limits():
    x = np.array([-1e4, -100.0, 0.0, 100.0, 1e4])
    for kind in ("silu", "gelu", "relu"):
        assert np.allclose(F.act(x, kind), [0, 0, 0, 100, 1e4], atol=1e-30)
        want0 = 0.0 if kind == "relu" else 0.5
        assert np.allclose(F.act_grad(x, kind), [0, 0, want0, 1, 1], atol=1e-30)


def test_gelu_is_the_tanh_form():
    x = np.linspace(-4, 12, 1001)
    assert np.allclose(F.act(x, "gelu"), gelu_tanh(x), rtol=1e-12, atol=1e-15)


def test_layernorm_of_a_constant_row_is_the_shift():
    y, mu, rs = F.layernorm(np.full((1, 9), 2.5), np.ones(9), np.arange(9.0))
    assert np.array_equal(y[0], np.arange(9.0)) and mu[0] == 2.5 and np.isclose(rs[0], 1e-5 ** -0.5)

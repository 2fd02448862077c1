"""The oracle's shares of scores that vanish: against the ratios written out with a common
factor taken out by hand, and against autograd (no GPU)."""
import numpy as np
import pytest
import torch

from oracle import moe_oracle as M


def test_equal_shares_far_down_and_nothing_for_infinite_masks():
    inf, low = np.inf, float(np.finfo(np.float32).min)
    l = np.array([[-100.0] * 4, [-1e4] * 4, [low] * 4, [-inf] * 4, [-inf, -300, -inf, -inf]])
    index = np.tile(np.arange(4, dtype=np.int32), (5, 1))
    for scoring in ("softmax", "sigmoid"):
        w = M.route_weights(l, index, scoring, True, 1.0)
        assert np.all(w[:3] == 0.25) and np.all(w[3] == 0) and w[4].tolist() == [0, 1, 0, 0]
        assert np.all(M.route_backward(np.arange(20.0).reshape(5, 4), l, index, scoring, True, 1.0)[3] == 0)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("level", [0.0, -3.0, -400.0, -2000.0])
def test_shares_and_their_gradient_against_autograd(scoring, level):
    g = np.random.default_rng(0)
    l, dw = level + g.standard_normal((7, 5)), g.standard_normal((7, 5))
    index = np.tile(np.arange(5, dtype=np.int32), (7, 1))
    index[2, 1], index[4] = -1, 5                    # never chosen
    live = torch.tensor((index >= 0) & (index < 5))
    x = torch.tensor(l, requires_grad=True)
    # shares by a softmax of the scores' logarithms
    logs = x if scoring == "softmax" else torch.nn.functional.logsigmoid(x)
    w = torch.softmax(logs.masked_fill(~live, -1e300), 1) * live
    (w * torch.tensor(dw)).sum().backward()
    assert np.allclose(M.chosen_shares(l, index, scoring), w.detach().numpy(), rtol=1e-11, atol=0)
    assert np.allclose(M.route_backward(dw, l, index, scoring, True, 1.0), x.grad.numpy(), rtol=1e-9, atol=1e-12)

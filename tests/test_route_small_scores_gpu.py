"""Renormalised logistic scores that are far below one: where every chosen logit is very
negative (a finite mask, a bias that chooses such experts) the weights are still their
scores' shares, and the gradient is that of these shares."""
import numpy as np
import pytest
import torch

from mxfp8_block_scaled_quantize_gb300 import binding
from tests.test_route_gpu import check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("level", [-20.0, -90.0, -100.0, -300.0, -1e4])
def test_logits_around_a_very_negative_level(level, t):
    g = torch.Generator().manual_seed(int(-level))
    l = (level + 2 * torch.randn(40, 64, generator=g)).to({"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}[t])
    dw = torch.randn(40, 6, generator=g).cuda()
    _, weight = check(l.cuda(), 6, t, scoring="sigmoid", dweight=dw, scale=2.5)
    # (a sum of six weights, each off by its division's half step, and the scale's)
    assert torch.all((weight.sum(1) - 2.5).abs() < 2.5 * 16 * 2.0 ** -24)


def test_equal_logits_share_alike_and_only_infinite_masks_get_nothing():
    inf, low = float("inf"), torch.finfo(torch.float32).min
    l = torch.zeros(6, 16)
    l[0], l[1], l[2], l[3], l[4] = -100.0, -1e4, low, -inf, -inf
    l[4, 5] = -200.0                                  # one left, far down
    l[5] = -inf
    l[5, ::2] = -150.0
    l = l.cuda()
    dw = torch.arange(24, device="cuda", dtype=torch.float32).view(6, 4)
    _, weight = check(l, 4, "fp32", scoring="sigmoid", dweight=dw)
    assert torch.all(weight[:3] == 0.25) and torch.all(weight[3] == 0) and torch.all(weight[5] == 0.25)
    assert weight[4].tolist() == [1, 0, 0, 0]


def test_a_bias_that_chooses_far_experts():
    l = torch.full((5, 32), -95.0)
    l[:, 0] = 50.0                                    # never chosen
    l[1:, 8:12] += torch.arange(4.0)
    l[2, 8] = -20.0                                   # one share is nearly all, the others vanish
    l[3, 9] = 3.0
    l[4, 8:12] = torch.tensor([-1.0, -0.1, -88.0, -0.01])
    l = l.cuda()
    bias = torch.zeros(32, device="cuda")
    bias[8:12] = 1e5
    index, weight = check(l, 4, "fp32", bias=bias, scoring="sigmoid", dweight=torch.rand(5, 4).cuda())
    assert torch.all(index.sort(1)[0] == torch.arange(8, 12, device="cuda")) and torch.all(weight[0] == 0.25)


def test_gradient_against_differences_far_down():
    g = torch.Generator().manual_seed(2)
    l = (-120 + torch.randn(4, 20, generator=g)).cuda()
    index = binding.route(l, 5, scoring="sigmoid")["index"]
    dw = torch.randn(4, 5, generator=g)
    d = binding.route_backward(dw.cuda(), l, index, scoring="sigmoid").cpu().double().numpy()
    at, base = index.cpu().numpy().astype(np.int64), l.cpu().double().numpy()

    def loss(v):
        s = 1 / (1 + np.exp(-np.take_along_axis(v, at, 1)))       # (e^-120 is a number in float64)
        return (s / s.sum(1, keepdims=True) * dw.double().numpy()).sum()

    for seed in range(3):
        v = np.random.default_rng(seed).standard_normal(base.shape)
        diff = (loss(base + 1e-5 * v) - loss(base - 1e-5 * v)) / 2e-5
        assert abs((d * v).sum() - diff) < 1e-6 + 300 * 2.0 ** -24 * np.abs(d * v).sum()

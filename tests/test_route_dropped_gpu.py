"""Choices dropped after the weights were made (an expert's capacity): the gradient of
the weights that were kept, which are shares of all the choices, comes from the forward
call's index and a gradient of 0 for what was dropped; checked against differences, and
all the way through sort, combine and combine's gradient."""
import numpy as np
import pytest
import torch

from mxfp8_block_scaled_quantize_gb300 import binding
from oracle import moe_oracle as M
from tests.test_route_gpu import HOW

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("how", HOW)
def test_gradient_of_kept_weights_against_differences(how):
    g = torch.Generator().manual_seed(4)
    tokens, experts, k, hidden = 12, 24, 4, 64
    logits = (2 * torch.randn(tokens, experts, generator=g)).cuda()
    o = binding.route(logits, k, scale=1.5, **how)
    chosen = o["index"]
    kept = chosen.clone()
    kept[::2, 1], kept[3, 0], kept[7] = -1, -1, -1
    s = binding.moe_sort(kept, experts)
    y = torch.randn(tokens * k, hidden, generator=g).cuda()
    dout = torch.randn(tokens, hidden, generator=g).cuda()
    dw = binding.moe_combine_backward(dout, y, s["row"], o["weight"])["dweight"]
    assert torch.all(dw[kept < 0] == 0)
    d = binding.route_backward(dw, logits, chosen, scale=1.5, **how).cpu().double().numpy()
    l, i, w = (v.cpu().double().numpy() for v in (logits, chosen, dw))
    i = i.astype(np.int64)
    # the loss is linear in the kept weights, whose gradients dw holds
    loss = lambda v: (M.route_weights(v, i, scale=1.5, **how) * w).sum()  # noqa: E731
    for seed in range(3):
        v = np.random.default_rng(seed).standard_normal(l.shape)
        diff = (loss(l + 1e-5 * v) - loss(l - 1e-5 * v)) / 2e-5
        # (differences: 1e-10 of third derivatives at most tens, and float64's rounding over 2e-5, of a loss of hundreds)
        assert abs((d * v).sum() - diff) < 1e-6 + 300 * 2.0 ** -24 * np.abs(d * v).sum()
    # a dropped choice's logit has a gradient too where the weights are shares of the choices
    if how["renormalise"]:
        assert abs(d[0, i[0, 1]]) > 1e-3 * np.abs(d[0]).max()


@pytest.mark.parametrize("how", HOW)
def test_an_index_outside_the_experts_is_a_choice_that_was_never_made(how):
    # weights as if the token had chosen the others alone: the gradient is theirs
    g = torch.Generator().manual_seed(6)
    logits = (2 * torch.randn(20, 16, generator=g)).cuda()
    index = binding.route(logits, 3, **how)["index"]
    dw = torch.randn(20, 3, generator=g).cuda()
    three = torch.cat([index, torch.full((20, 1), -1, dtype=torch.int32, device="cuda")], 1)
    d = binding.route_backward(torch.cat([dw, torch.ones(20, 1, device="cuda")], 1), logits, three, **how)
    assert torch.equal(d, binding.route_backward(dw, logits, index, **how))

"""Choices among 16-bit logits without a bias, whose keys share a word with their index:
ties, -0, masks, infinities, NaN and the type's lowest value, for numbers of choices on
either side of where a lane sorts its keys first (half of the experts that it holds)."""
import numpy as np
import pytest
import torch

from mxfp8_block_scaled_quantize_gb300 import binding
from oracle import moe_oracle as M
from tests.test_layernorm_gpu import T
from tests.test_route_gpu import check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("experts,k", [(8, 1), (8, 8), (40, 1), (64, 7), (100, 1), (128, 2), (128, 8), (200, 3), (256, 4), (256, 5),
                                       (500, 7), (512, 8), (512, 32), (1024, 15), (1000, 16)])
@pytest.mark.parametrize("t", ["bf16", "fp16"])
def test_ties_masks_nan_and_infinities(experts, k, t):
    inf, low = float("inf"), torch.finfo(T[t]).min
    g = torch.Generator().manual_seed(experts + k)
    l = torch.randn(14, experts, generator=g)
    l[1] = 0.0                                        # ties everywhere
    l[2, ::2] = -0.0
    l[2, 1::2] = 0.0
    l[3] = torch.randint(-2, 3, (experts,), generator=g).float()          # ties in classes
    l[4] = -inf
    l[5] = -inf
    l[5, experts // 2:] = low                         # masks of both kinds
    l[6] = low
    l[6, experts - 1] = -1.0
    l[7] = -l[0].abs()                                # negative numbers alone
    l[8] = torch.randint(-2, 3, (experts,), generator=g).float() * 2.0 ** -24      # subnormal, in fp16
    l[9] = torch.finfo(T[t]).max
    finite = 10
    l[10, ::3] = inf
    l[11, ::3] = float("nan")
    l[12] = float("nan")
    l[13, ::2], l[13, 1::2] = float("nan"), -inf
    l = l.to(T[t]).cuda()
    o = binding.route(l, k)
    assert np.array_equal(o["index"].cpu().numpy(), M.route_index(l.float().cpu().numpy(), k))
    assert torch.isnan(o["weight"][12]).all()
    dw = torch.randn(finite, k, generator=g).cuda()
    for scoring in ("softmax", "sigmoid"):
        for renormalise in (True, False):
            check(l[:finite], k, t, scoring=scoring, renormalise=renormalise, dweight=dw)

"""LayerNorm forward and backward on rows of up to 2^24 elements, which a block
reads from memory more than once, against the float64 oracle.  Terms of one sign
and nearly one size: added one after another in a thread (65536 of them) they
lose up to a thousandth, which the small spread of such a row turns into errors
far outside the bounds of the chain that the kernels promise."""
import numpy as np
import pytest
import torch

from mxfp8_block_scaled_quantize_gb300 import binding
from oracle import ffn_oracle as F
from tests.test_layernorm_gpu import T, assert_within, f64

pytestmark = pytest.mark.gpu


def depth(hidden):
    # eight terms of a tree, 64 trees of a batch, the batches of a thread (256 of
    # them, 512 terms to a batch), five butterfly levels, eight warps
    return 3 + 64 + -(-hidden // (256 * 512)) + 5 + 8


@pytest.mark.parametrize("hidden", [70001, (1 << 17) + 1, (1 << 20) - 1, 1 << 24])
@pytest.mark.parametrize("t,tp", [("fp32", "fp32"), ("bf16", "bf16"), ("fp16", "fp32")])
def test_sums_of_long_rows(hidden, t, tp):
    g = torch.Generator().manual_seed(hidden)
    x = torch.full((1, hidden), 1.1)
    x[:, ::997] += 1e-2 * torch.randn(1, -(-hidden // 997), generator=g)
    sign = torch.where(torch.rand(1, hidden, generator=g) < 0.5, -1.0, 1.0)
    x, ga = x.to(T[t]).cuda(), torch.full((hidden,), 0.7).to(T[tp]).cuda()
    o = binding.layernorm(x, ga)
    binding.te_mx_device_status()
    xv, gv = f64(x), f64(ga)
    want, wmu, wrs = F.layernorm(xv, gv)
    d = depth(hidden)
    dmu, rho = F.layernorm_stat_bounds(xv, 1e-5, d)
    assert_within(f64(o["mu"]), wmu, dmu, "mu")
    assert_within(f64(o["rsigma"]), wrs, rho * wrs, "rsigma")
    assert_within(f64(o["y"]), want, F.layernorm_bound(xv, gv, 0.0, 1e-5, d, t), "y")
    # backward: a spread row, dy of one sign, then dy of the sign of xh
    x = (torch.randn(1, hidden, generator=g).abs() * sign + 0.3).to(T[t]).cuda()
    mu, rs = (torch.tensor([v], device="cuda") for v in (0.3, 0.9))
    for dy in (torch.full((1, hidden), 0.13), 0.13 * sign):
        dy = dy.to(T[t]).cuda()
        got = binding.layernorm_backward(dy, x, ga, mu, rs)
        binding.te_mx_device_status()
        args = [f64(v) for v in (dy, x, ga, mu, rs)]
        bounds = F.layernorm_backward_bounds(*args, d, 1 + 32 + 38 + 8, t, tp)
        for k, w, b in zip(("dx", "dgamma", "dbeta"), F.layernorm_backward(*args), bounds):
            assert_within(f64(got[k]).reshape(w.shape), w, b, k)

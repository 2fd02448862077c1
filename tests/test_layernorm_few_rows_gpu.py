"""LayerNorm backward around the limit between its kernels for few and for many
rows on 16-byte boundaries, against the float64 oracle within its bounds: on both
sides in rows and row lengths, in place (where the one-launch kernel may not be
used), single outputs, repeated calls."""
import pytest
import torch

from mxfp8_block_scaled_quantize_gb300 import binding
from oracle import ffn_oracle as F
from tests import test_layernorm_gpu as L

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,hidden,t,tp,pad", [
    (2, 8, "bf16", "bf16", 0), (304, 64, "bf16", "fp32", 8), (305, 64, "bf16", "fp32", 0), (512, 1024, "bf16", "bf16", 0),
    (513, 1024, "bf16", "bf16", 24), (1000, 2048, "fp16", "fp32", 0), (1030, 2048, "fp16", "fp16", 0),
    (304, 16384, "fp32", "fp32", 0), (305, 16384, "fp32", "fp32", 0), (1000, 7168, "bf16", "fp32", 8),
    (3200, 7168, "bf16", "bf16", 0), (3600, 7168, "bf16", "bf16", 0), (900, 4096, "fp32", "fp32", 4),
    (20, 20480, "bf16", "bf16", 0), (310, 16392, "bf16", "bf16", 0), (7, 40960, "fp16", "fp16", 0)])
def test_backward(rows, hidden, t, tp, pad):
    x, dy, ga, be = L.make(rows, hidden, t, tp, 5 * rows + hidden, pad)
    o = binding.layernorm(x, ga, be)
    mu, rs = o["mu"], o["rsigma"]
    dx, dga, dbe = L.check_backward(dy, x, ga, mu, rs, t, tp, pad)
    for _ in range(3):
        again = binding.layernorm_backward(dy, x, ga, mu, rs)
        assert torch.equal(again["dx"], dx) and torch.equal(again["dgamma"], dga) and torch.equal(again["dbeta"], dbe)
    alone = binding.layernorm_backward(dy, x, ga, mu, rs, dparams=False)
    args = [L.f64(v) for v in (dy, x, ga, mu, rs)]
    want = F.layernorm_backward(*args)
    bounds = F.layernorm_backward_bounds(*args, L.row_sum_depth(hidden), L.column_sum_depth(rows), t, tp)
    L.assert_within(L.f64(alone["dx"]), want[0], bounds[0], "dx alone")
    for over in (dy, x):                                  # dx over dy, and over x
        d = {id(dy): dy.clone(), id(x): x.clone()}
        o = binding.layernorm_backward(d[id(dy)], d[id(x)], ga, mu, rs, out={"dx": d[id(over)]})
        for got, w, b, name in zip((o["dx"], o["dgamma"], o["dbeta"]), want, bounds, ("dx", "dgamma", "dbeta")):
            L.assert_within(L.f64(got), w, b, name + " in place")

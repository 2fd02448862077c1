"""LayerNorm of many rows off 16-byte boundaries: the persistent kernels take
several rows per group of threads, load one ahead and join the columns' sums.
Every number of elements per thread, more and fewer rows than groups, in place,
repeated, and row lengths on both sides of each kernel's limit."""
import pytest
import torch

from mxfp8_block_scaled_quantize_gb300 import binding
from tests import test_layernorm_gpu as L

pytestmark = pytest.mark.gpu


def copy(x, pad, offset):
    """x in a buffer of the same layout (which chooses the kernel, and so the order of the sums)."""
    v, _ = L.guarded(*x.shape, x.shape[1] + pad, x.dtype, offset)
    return v.copy_(x)


@pytest.mark.parametrize("rows,hidden,t,tp,pad,offset", [
    (3000, 1023, "fp16", "fp32", 2, 0), (5000, 65, "bf16", "fp32", 0, 0), (6000, 31, "bf16", "bf16", 0, 1),
    (1000, 333, "fp32", "fp32", 1, 3), (700, 2047, "bf16", "bf16", 1, 1), (700, 2049, "fp16", "fp16", 0, 0),
    (151, 2051, "fp32", "fp32", 0, 0), (320, 4095, "bf16", "fp32", 0, 5), (320, 4097, "bf16", "bf16", 3, 0),
    (400, 5003, "fp32", "fp32", 0, 0), (200, 8191, "fp16", "fp32", 0, 0), (200, 8193, "bf16", "bf16", 0, 0),
    (170, 16383, "bf16", "bf16", 0, 0), (400, 16384, "bf16", "fp32", 1, 0), (3, 1023, "bf16", "bf16", 0, 0),
    (4097, 1, "fp32", "fp32", 0, 0), (2000, 512, "bf16", "bf16", 0, 1)])
def test_forward_and_backward(rows, hidden, t, tp, pad, offset):
    x, dy, ga, be = L.make(rows, hidden, t, tp, rows + 3 * hidden, pad, offset)
    mu, rs, y = L.check_forward(x, ga, be, t, pad, offset)
    dx, dga, dbe = L.check_backward(dy, x, ga, mu, rs, t, tp, pad, offset)
    for _ in range(3):                                    # the same bits each time, and in place
        d, v = copy(dy, pad, offset), copy(x, pad, offset)
        o = binding.layernorm_backward(d, x, ga, mu, rs, out={"dx": d})
        again = [binding.layernorm(v, ga, be, out={"y": v})["y"], o["dx"], *binding.layernorm_backward(dy, x, ga, mu, rs).values()]
        for a, b in zip(again, (y, dx, dx, dga, dbe)):
            assert torch.equal(a, b)
    o = binding.layernorm_backward(dy, x, ga, mu, rs, dparams=False)
    assert torch.equal(o["dx"], dx)
    assert torch.equal(binding.layernorm(x, ga, None, stats=False)["y"],
                       binding.layernorm(x, ga, torch.zeros_like(ga))["y"])

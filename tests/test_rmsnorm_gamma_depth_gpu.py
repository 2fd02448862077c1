"""RMSNorm's gamma gradient over many rows of rows that no block holds: the kernel has few
partial sums there, and its chains stay within the depth that the tests' bound states."""
import numpy as np
import pytest
import torch

from mxfp8_block_scaled_quantize_gb300 import binding
from oracle import moe_oracle as M
from tests.test_layernorm_gpu import f64
from tests.test_rmsnorm_gpu import check_backward, column_depth, make

pytestmark = pytest.mark.gpu


def test_long_rows_of_many_rows_within_the_stated_chain():
    x, res, dy, dz, ga = make(3000, 8201, "bf16", "fp32", 5)
    rs = binding.rmsnorm(x, ga)["rsigma"]
    check_backward(dy, x, ga, rs, dz, "bf16", "fp32")


def test_one_partial_sum_of_a_thousand_rows():
    # so long rows that a block per part of the columns fills the GPU: all rows in one sum.  Every
    # term is 2^-15 - 2^-20 above one, which a single chain loses past 512 (half a step there)
    rows = 1024
    hidden = (16 * torch.cuda.get_device_properties(0).multi_processor_count + 1) * 512 + 16
    one = torch.ones(rows, hidden, dtype=torch.bfloat16, device="cuda")
    term = 1 + 2.0 ** -15 - 2.0 ** -20
    rs = torch.full((rows,), term, device="cuda")
    ga, dga = torch.ones(hidden, device="cuda"), torch.empty(hidden, device="cuda")
    ws = torch.empty(binding.te_mx_rmsnorm_backward_workspace_size(rows, hidden), dtype=torch.uint8, device="cuda")
    binding.te_mx_rmsnorm_backward(one.data_ptr(), hidden, one.data_ptr(), hidden, rows, hidden, binding.BF16, ga.data_ptr(),
                                   binding.FP32, rs.data_ptr(), 0, 0, 0, 0, dga.data_ptr(), ws.data_ptr(), ws.numel(), 0)
    binding.te_mx_device_status()
    exact, u = rows * term, 2.0 ** -24
    bound = M.MORE * (column_depth(rows) + 3) * u * exact + u * exact      # the sum's chain; one rounding
    assert np.abs(f64(dga) - exact).max() <= bound

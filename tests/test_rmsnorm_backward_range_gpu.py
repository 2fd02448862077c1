"""RMSNorm's gradient at the end of its range: rows whose 1/sigma squared is no fp32
number."""
import pytest
import torch

from mxfp8_block_scaled_quantize_gb300 import binding
from tests.test_layernorm_gpu import T
from tests.test_rmsnorm_gpu import check_backward, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [40, 700])            # one launch, the ring
@pytest.mark.parametrize("hidden", [512, 2048, 515])
@pytest.mark.parametrize("t", ["fp32", "bf16"])
def test_a_tiny_epsilon_and_rows_of_zeros_or_tiny_values(rows, hidden, t):
    _, _, dy, dz, ga = make(rows, hidden, t, t, rows + hidden)
    z = torch.randn(rows, hidden, generator=torch.Generator().manual_seed(3)) * 1e-20
    z[::3] = 0
    z = z.to(T[t]).cuda()
    rs = binding.rmsnorm(z, ga, eps=1e-40)["rsigma"]
    assert torch.isfinite(rs).all() and torch.isinf(rs * rs).all()
    check_backward(dy, z, ga, rs, dz, t, t)
    check_backward(dy, z, ga, rs, None, t, t)

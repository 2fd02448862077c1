"""te_mx_layernorm_backward's partial sums stay inside the workspace that its size
function names, whatever the GPU's SM count: rows around the number of partial
sums per column, every kernel that leaves some; bytes past the workspace kept."""
import pytest
import torch

from mxfp8_block_scaled_quantize_gb300 import binding
from tests.test_layernorm_gpu import column_sum_depth

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [1, 151, 152, 153, 303, 304, 305, 609, 5000])
@pytest.mark.parametrize("hidden,t", [(64, torch.bfloat16), (1000, torch.float16), (1023, torch.float16), (20000, torch.bfloat16),
                                      (9001, torch.float32), (16384, torch.float32)])
def test_partial_sums_stay_in_the_workspace(rows, hidden, t):
    g = torch.Generator(device="cuda").manual_seed(rows + hidden)
    x, dy = (torch.randn(rows, hidden, generator=g, device="cuda").to(t) for _ in range(2))
    ga = torch.ones(hidden, dtype=t, device="cuda")
    mu, rs = x.float().mean(1), torch.ones(rows, device="cuda")
    need = binding.te_mx_layernorm_backward_workspace_size(rows, hidden)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert need <= 2 * max(sms, 152) * 2 * hidden * 4 and need == min(rows, need // (8 * hidden)) * 8 * hidden
    ws = torch.full((need + (sms + 8) * 8 * hidden,), 0xA5, dtype=torch.uint8, device="cuda")
    over = dy.clone()                                      # dx in dy's place: the persistent kernels at every row count
    o = binding.layernorm_backward(over, x, ga, mu, rs, out={"dx": over}, workspace=ws[:need])
    torch.cuda.synchronize()
    binding.te_mx_device_status()
    assert torch.all(ws[need:] == 0xA5)
    want = dy.double().sum(0)
    bound = column_sum_depth(rows) * 2.0 ** -24 * dy.double().abs().sum(0)
    assert torch.all((o["dbeta"].double() - want).abs() <= bound + torch.finfo(t).eps / 2 * (want.abs() + bound))

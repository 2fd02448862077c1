"""te_mx_gated_backward with many rounds per block: a block walks strips of 64
rows x 512 columns and gathers a strip's row-wise scale bytes in one of four
slots, so the slots are used again from the fifth round on.  Ten rounds and more
per block, with strips that fill the width and with a cut last strip that a block
meets in every round (the strips of a band divide the GPU's SMs), where most of
the block's warps own no unit.  The quantised copies bit for bit against those
that te_mx_quantize makes of the bf16 gradient, and the oracle's at both ends."""
import numpy as np
import pytest
import torch

from mxfp8_block_scaled_quantize_gb300 import binding
from oracle import mx_oracle as O
from tests import _util as U

pytestmark = pytest.mark.gpu

ROUNDS = 10


def rows_for(n):
    """Rows whose strips give every SM's block ROUNDS rounds of width n."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    strips_per_band = -(-n // 512)
    return 64 * -(-sms * ROUNDS // strips_per_band)


def make(rows, n, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    spread = torch.exp2(16 * torch.rand(rows, 1, generator=g, device="cuda") - 20)         # scale bytes that differ by row
    dh = (torch.randn(rows, n, generator=g, device="cuda") * spread).to(torch.bfloat16)
    gu = (torch.randn(rows, 2 * n, generator=g, device="cuda") * 2).to(torch.bfloat16)
    return dh, gu


# 64, 96: one cut strip per band; 768, 3840: the last of two and of eight strips
# cut; 544, 1056: a single unit of 32 columns in it; 512, 1024: no strip cut
@pytest.mark.parametrize("dense,colwise", [(False, True), (True, True), (False, False), (True, False)])
@pytest.mark.parametrize("n", [64, 96, 544, 768, 1056, 3840, 512, 1024])
def test_scale_slots_used_again(n, dense, colwise):
    rows = rows_for(n) - 3                                 # (a ragged last band)
    dh, gu = make(rows, n, n)
    d = binding.gated_backward(dh, gu, dense=True, rowwise=False, colwise=False)["d_gate_up"]
    o = binding.gated_backward(dh, gu, dense=dense, rowwise=True, colwise=colwise)
    torch.cuda.synchronize()
    binding.te_mx_device_status()
    if dense:
        assert torch.equal(o["d_gate_up"], d)
    want = binding.quantize(d)
    blocks = 2 * n // 32
    assert torch.equal(o["q_row"], want["q_row"]), "row-wise codes"
    assert torch.equal(o["s_row"][:, :blocks], want["s_row"][:, :blocks]), "row-wise scales"
    for part in (slice(0, 64), slice(rows - 64, rows)):
        q, s = O.quantize_rowwise(U.bf16_bits(d[part].contiguous()))
        U.assert_bytes_equal(o["q_row"][part].cpu().numpy(), q, "row-wise codes")
        U.assert_bytes_equal(np.ascontiguousarray(o["s_row"][part, :blocks].cpu().numpy()), s, "row-wise scales")
    if colwise:
        kp = -(-rows // 128) * 128
        padded = torch.zeros(kp, 2 * n, dtype=torch.bfloat16, device="cuda")
        padded[:rows] = d
        want = binding.quantize(padded, rowwise=False, colwise=True)
        assert torch.equal(o["q_col"], want["q_col"]), "column-wise codes"
        assert torch.equal(o["s_col"][:, :kp // 32], want["s_col"][:, :kp // 32]), "column-wise scales"


def test_repeats_bit_for_bit():
    n = 768
    dh, gu = make(rows_for(n), n, 5)
    a = binding.gated_backward(dh, gu)
    for _ in range(8):
        b = binding.gated_backward(dh, gu)
        for k in ("q_row", "q_col"):
            assert torch.equal(a[k], b[k]), k
        assert torch.equal(a["s_row"][:, :2 * n // 32], b["s_row"][:, :2 * n // 32])
    torch.cuda.synchronize()
    binding.te_mx_device_status()

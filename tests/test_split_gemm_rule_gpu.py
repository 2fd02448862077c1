"""te_mx_gemm with 64 to 128 tokens and few K-steps, on both sides of the rule that
picks tiles with K split over clusters or the larger ones: tokens 64 / 65 / 96 / 97
/ 128, a quarter, one and two tiles of 128 columns per SM, 27 and 28 K-steps.
Against the float64 oracle within the GEMM's bound; equal bits from run to run."""
import numpy as np
import pytest
import torch

from mxfp8_block_scaled_quantize_gb300 import binding
from oracle import mx_oracle as O
from tests import _util as U
from tests import test_gated_gemm_gpu as G

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,K,bias", [
    (64, 8192, 2048, True), (65, 8192, 2048, True), (65, 4864, 2176, False), (128, 4864, 2048, True), (128, 4880, 2048, True),
    (96, 19456, 2048, False), (97, 19456, 2048, True), (97, 19472, 2048, False), (128, 38912, 2048, True),
    (96, 38928, 2048, True), (128, 38928, 2048, False), (100, 8208, 3456, True), (100, 8208, 3584, True),
])
def test_both_sides_of_the_rule(M, N, K, bias):
    qa, sa = G.operand(M, K, M + K, outliers=True)
    qb, sb = G.operand(N, K, N + K, std=0.05)
    b = torch.randn(N, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16) if bias else None
    d, buf = U.guarded_bf16(M, N)
    args = (*G.upload(qa, sa), *G.upload(qb, sb))
    binding.gemm(*args, bias=None if b is None else b.cuda(), out=(d, None))
    binding.te_mx_device_status()
    U.check_guard(buf, M * N)
    ref = O.mx_gemm(qa, sa, qb, sb, None if b is None else U.bf16_bits(b))
    bad = ~(np.abs(G.f64(d) - ref["d"]) <= O.gemm_error_bound(ref["d"], ref["sigma"]))
    assert not bad.any(), f"{int(bad.sum())} of {bad.size} outside the bound, first {tuple(np.argwhere(bad)[0])}"
    again, _ = binding.gemm(*args, bias=None if b is None else b.cuda())
    assert torch.equal(again, d)

"""te_mx_gemm and te_mx_gated_gemm where K is split over clusters: few tokens or
few output tiles.  Against the float64 oracle within the GEMM's bound, single
tokens to several token blocks, widths that fill no tile, K whose scale groups
divide unevenly over the blocks, with and without bias; equal bits from run to
run; scale-pitch padding 0xFF, canary tails."""
import numpy as np
import pytest
import torch

from mxfp8_block_scaled_quantize_gb300 import binding
from oracle import mx_oracle as O
from tests import _util as U
from tests import test_gated_gemm_gpu as G

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,K,bias", [
    (1, 16, 2048, False), (1, 7168, 2048, True), (3, 144, 2176, True), (16, 1040, 4096, False), (17, 128, 3840, True),
    (31, 2064, 2560, False), (64, 272, 8192, True), (100, 1008, 2048, False), (128, 128, 4224, True), (129, 400, 2048, True),
    (200, 1024, 4096, False), (255, 256, 2944, True), (256, 1040, 2048, True), (300, 528, 6144, False), (1000, 1024, 2048, True),
    (700, 2000, 2176, False),
])
def test_plain(M, N, K, bias):
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
    for _ in range(3):
        again, _ = binding.gemm(*args, bias=None if b is None else b.cuda())
        assert torch.equal(again, d)


@pytest.mark.parametrize("M,n,K,kind,bias,aux", [
    (129, 336, 2176, "silu", True, True), (300, 144, 1024, "gelu", False, True), (1000, 512, 512, "silu", False, True),
    (256, 1024, 4096, "relu", True, False), (700, 208, 384, "silu", True, True),
])
def test_gated_with_several_token_blocks(M, n, K, kind, bias, aux):
    G.check(M, n, K, kind, bias, aux, M + n)


def test_nan_scales_stay_in_their_rows_and_columns():
    qa, sa = G.operand(40, 2048, 1)
    qb, sb = G.operand(96, 2048, 2)
    clean, _ = binding.gemm(*G.upload(qa, sa), *G.upload(qb, sb))
    qa[7, 64:96], sa[7, 2] = 0x7F, 0xFF
    qb[50, 2016:], sb[50, 63] = 0x7F, 0xFF
    d, _ = binding.gemm(*G.upload(qa, sa), *G.upload(qb, sb))
    bad = torch.zeros(40, 96, dtype=torch.bool)
    bad[7], bad[:, 50] = True, True
    assert torch.equal(torch.isnan(d.cpu()), bad) and torch.equal(d.cpu()[~bad], clean.cpu()[~bad])


def test_in_a_graph_and_on_another_stream():
    args = (*G.upload(*G.operand(5, 4096, 3)), *G.upload(*G.operand(512, 4096, 4)))
    want, _ = binding.gemm(*args)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        a, _ = binding.gemm(*args)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b, _ = binding.gemm(*args)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, want) and torch.equal(b, want)

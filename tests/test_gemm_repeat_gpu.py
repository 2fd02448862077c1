"""MXFP8 GEMMs add in an order that depends on the shapes alone: repeated calls,
other work between them, give the same bits, at short and long K, with every
epilogue, dense and grouped."""
import pytest
import torch

import mxfp8_block_scaled_quantize_gb300 as temx
from tests import test_gated_gemm_gpu as G

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M, N, K", [(200, 384, 4096), (1500, 1040, 1024), (1500, 2064, 4224), (4096, 2048, 7168)])
def test_dense(M, N, K):
    a, b = G.upload(*G.operand(M, K, 1)), G.upload(*G.operand(N, K, 2))
    g = torch.Generator(device="cuda").manual_seed(3)
    bias = torch.randn(N, generator=g, device="cuda").to(torch.bfloat16)
    pre = torch.randn(M, N, generator=g, device="cuda").to(torch.bfloat16)
    calls = [lambda: temx.gemm(*a, *b)[0], lambda: temx.gemm(*a, *b, bias=bias, gelu=True)[1],
             lambda: temx.gemm(*a, *b, dgelu_aux=pre)[0],
             lambda: temx.gemm(*a, *b, accumulate=torch.zeros(M, N, device="cuda"))[0]]
    for f in calls:
        want = f()
        for _ in range(12):
            torch.randn(1 << 22, device="cuda")
            assert torch.equal(f(), want)
    temx.te_mx_device_status()


def test_grouped():
    sizes, N, K = [700, 0, 513, 900, 300], 512, 2176
    a, (qw, sw) = G.upload(*G.operand(sum(sizes), K, 4)), G.upload(*G.operand(len(sizes) * N, K, 5))
    m = torch.tensor(sizes, dtype=torch.int32, device="cuda")
    f = lambda: temx.grouped_gemm(m, *a, qw.view(len(sizes), N, K), sw, gelu=True)  # noqa: E731
    want = f()
    for _ in range(12):
        got = f()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    temx.te_mx_device_status()

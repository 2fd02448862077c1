"""Grouped gated GEMM around the limit between its kernels: few tokens (K split
over clusters, the groups' blocks of tokens found on the device) and more, in few
and many groups, empty ones, blocks of 128 tokens exactly full and one over, rows
past the groups' sum, against the float64 oracle."""
import pytest
import torch

from mxfp8_block_scaled_quantize_gb300 import binding
from tests import test_gated_gemm_gpu as G

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sizes,n,K,kind,bias,aux,total", [
    ([1], 16, 128, "silu", True, True, None), ([0, 0, 1], 272, 4096, "gelu", True, True, None),
    ([1, 2, 0, 1, 4], 768, 4096, "silu", False, False, 40), ([0] * 1000 + [3] + [0] * 20 + [2, 1, 0], 48, 640, "silu", True, True, None),
    ([128], 64, 1024, "relu", True, True, None), ([129], 80, 1024, "silu", False, True, None),
    ([127, 1, 128, 129], 144, 2048, "gelu", True, True, 400), ([300, 0, 212], 208, 1536, "silu", True, True, None),
    ([300, 0, 213], 208, 1536, "silu", True, True, None), ([8] * 64, 512, 512, "silu", True, True, None),
    ([8] * 63 + [9], 1040, 384, "relu", False, True, None), ([700, 0, 65, 400], 144, 2048, "silu", True, True, 1300)])
def test_sizes(sizes, n, K, kind, bias, aux, total):
    G.check_grouped(sizes, n, K, kind, bias, aux, sum(sizes) + n + K, total)


def test_sizes_that_change_in_a_graph():
    sizes = torch.tensor([3, 0, 5, 2], dtype=torch.int32, device="cuda")
    (qx, sx), (qw, sw) = G.upload(*G.operand(10, 2048, 1)), G.upload(*G.operand(4 * 2 * 96, 2048, 2))
    qw = qw.view(4, 192, 2048)
    want = {}
    for m in ((3, 0, 5, 2), (0, 10, 0, 0), (1, 1, 1, 7)):
        h, _ = binding.grouped_gated_gemm(torch.tensor(m, dtype=torch.int32, device="cuda"), qx, sx, qw, sw)
        want[m] = h.clone()
    out = torch.empty(10, 96, dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        binding.grouped_gated_gemm(sizes, qx, sx, qw, sw, out=(out, None))
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            binding.grouped_gated_gemm(sizes, qx, sx, qw, sw, out=(out, None))
    for m, w in list(want.items()) * 2:
        sizes.copy_(torch.tensor(m, dtype=torch.int32))
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, w)
    binding.te_mx_device_status()

"""The helpers' ``stream`` argument: work, outputs and temporaries belong to that
stream, also while the current stream is busy and takes memory meanwhile."""
import pytest
import torch

import mxfp8_block_scaled_quantize_gb300 as temx
from tests import test_gated_gemm_gpu as G

pytestmark = pytest.mark.gpu


def same(a, b):
    if isinstance(a, dict):
        return a.keys() == b.keys() and all(same(a[k], b[k]) for k in a)
    if isinstance(a, tuple):
        return all(same(x, y) for x, y in zip(a, b))
    return a is b is None or torch.equal(a, b)


def test_stream_argument():
    g = torch.Generator().manual_seed(1)
    x = torch.randn(700, 2048, generator=g).to(torch.bfloat16).cuda()
    dy = torch.randn(700, 2048, generator=g).to(torch.bfloat16).cuda()
    ga, be = torch.rand(2, 2048, generator=g).to(torch.bfloat16).cuda()
    args = (*G.upload(*G.operand(700, 1024, 2)), *G.upload(*G.operand(512, 1024, 3)))
    experts = torch.tensor([300, 400], dtype=torch.int32, device="cuda")
    gw, gsw = G.upload(*G.operand(2 * 512, 1024, 4))
    fwd = temx.layernorm(x, ga, be)
    pre = temx.gated_gemm(*args, aux=True)[1]
    dh = torch.randn(700, 256, generator=g).to(torch.bfloat16).cuda()
    calls = [lambda **k: temx.layernorm(x, ga, be, **k),
             lambda **k: temx.layernorm_backward(dy, x, ga, fwd["mu"], fwd["rsigma"], **k),
             lambda **k: temx.gated_gemm(*args, aux=True, **k),
             lambda **k: temx.grouped_gated_gemm(experts, *args[:2], gw.view(2, 512, 1024), gsw, aux=True, **k),
             lambda **k: temx.gated_backward(dh, pre, dense=True, rowwise=False, colwise=False, **k)]
    want = [f() for f in calls]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for f, w in zip(calls, want):
        got = []
        for _ in range(8):
            got.append(f(stream=s))
            for n in (1 << 12, 1 << 20, 5 << 20):          # what the current stream takes meanwhile
                torch.empty(n, dtype=torch.uint8, device="cuda").fill_(0xFF)
        torch.cuda.synchronize()
        assert all(same(r, w) for r in got)
    temx.te_mx_device_status()

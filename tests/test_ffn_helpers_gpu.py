"""What the LayerNorm and gated helpers refuse before anything is launched: buffers
and operands of other sizes, types, layouts or devices than the call's."""
import pytest
import torch

import mxfp8_block_scaled_quantize_gb300 as temx

pytestmark = pytest.mark.gpu

M, H, K, F = 40, 64, 128, 32


def zeros(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype, device="cuda")


def u8(*shape):
    return zeros(*shape, dtype=torch.uint8)


def f32(*shape):
    return zeros(*shape, dtype=torch.float32)


def calls():
    x, g = zeros(M, H), zeros(H)
    ln = lambda **k: temx.layernorm(k.pop("x", x), k.pop("g", g), k.pop("b", None), **k)  # noqa: E731
    bwd = lambda **k: temx.layernorm_backward(k.pop("dy", x), x, g, k.pop("mu", f32(M)), k.pop("rs", f32(M)), **k)  # noqa: E731
    gated = lambda **k: temx.gated_gemm(k.pop("q", u8(M, K)), k.pop("s", u8(M, 16)), u8(2 * F, K),  # noqa: E731
                                        k.pop("sw", u8(2 * F, 16)), **k)
    moe = lambda **k: temx.grouped_gated_gemm(k.pop("m", torch.tensor([M, 0], dtype=torch.int32, device="cuda")),  # noqa: E731
                                              u8(M, K), k.pop("s", u8(M, 16)), k.pop("w", u8(2, 2 * F, K)),
                                              k.pop("sw", u8(4 * F, 16)), **k)
    db = lambda **k: temx.gated_backward(k.pop("dh", zeros(M, F)), k.pop("gu", zeros(M, 2 * F)), **k)  # noqa: E731
    return {
        "ln": [ln, [dict(x=x.double()), dict(x=x.t()), dict(x=x.cpu()), dict(g=zeros(H + 1)), dict(g=g.cpu()),
                    dict(g=zeros(2 * H)[::2]), dict(b=f32(H)), dict(b=zeros(H - 1)), dict(out={"y": zeros(M, H + 8)}),
                    dict(out={"y": f32(M, H)}), dict(out={"mu": f32(M - 1), "rsigma": f32(M)}),
                    dict(out={"mu": f32(M), "rsigma": zeros(M)})]],
        "ln_bwd": [bwd, [dict(dy=f32(M, H)), dict(dy=zeros(M - 1, H)), dict(mu=f32(M - 1)), dict(rs=zeros(M)),
                         dict(rs=f32(2 * M)[::2]), dict(out={"dx": zeros(M, H - 8)}),
                         dict(out={"dgamma": zeros(H - 1), "dbeta": zeros(H)}),
                         dict(out={"dgamma": zeros(H), "dbeta": f32(H)})]],
        "gated": [gated, [dict(q=u8(K, M).t()), dict(q=zeros(M, K)), dict(s=u8(M - 1, 16)), dict(s=f32(M, 16)),
                          dict(sw=u8(F, 16)), dict(bias=zeros(F)), dict(bias=f32(2 * F)), dict(bias=zeros(4 * F)[::2]),
                          dict(q=u8(M, K).cpu()), dict(out=(zeros(M, 2 * F), None)), dict(out=(zeros(M, F), zeros(M, F))),
                          dict(out=(f32(M, F), None)), dict(out=(zeros(F, M).t(), None))]],
        "moe": [moe, [dict(m=torch.zeros(2, dtype=torch.int64, device="cuda")), dict(m=torch.zeros(2, dtype=torch.int32)),
                      dict(m=zeros(3, dtype=torch.int32)), dict(s=u8(M - 1, 16)), dict(w=u8(2, 2 * F, 2 * K)),
                      dict(sw=u8(2 * F, 16)), dict(bias=zeros(2, F)), dict(out=(zeros(M, 2 * F), None))]],
        "gated_bwd": [db, [dict(dh=f32(M, F)), dict(gu=zeros(M, F)), dict(dh=zeros(F, M).t()), dict(gu=zeros(M - 1, 2 * F)),
                           dict(out={"q_row": u8(M, F), "s_row": u8(M, 16)}), dict(out={"q_row": u8(M, 2 * F), "s_row": u8(1, 16)}),
                           dict(out={"q_col": u8(F, 128), "s_col": u8(F, 16)}),
                           dict(dense=True, out={"d_gate_up": f32(M, 2 * F)})]],
    }


@pytest.mark.parametrize("op", ["ln", "ln_bwd", "gated", "moe", "gated_bwd"])
def test_helper_refusals(op):
    call, bad = calls()[op]
    call()                                               # (the arguments that each bad call changes are right)
    for i, kw in enumerate(bad):
        with pytest.raises((AssertionError, TypeError, temx.TemxError)):
            call(**kw)
            raise RuntimeError(f"{op}: bad call {i} was taken")
    torch.cuda.synchronize()
    temx.te_mx_device_status()

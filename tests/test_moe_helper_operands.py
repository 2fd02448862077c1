"""What the RMSNorm, router, sorting, dispatch and combine helpers refuse before
they call the library, on the CPU: stand-ins that say they are on a CUDA device
take the tensors' places and a recorder the library's, so a call that would hand it
a CPU tensor's address is seen, and nothing runs."""
import pytest
import torch

from mxfp8_block_scaled_quantize_gb300 import binding
from tests.test_ffn_helper_operands import Cuda, Recorder, each_moved, f32, u8, zeros

M, H, E, K, R = 64, 128, 8, 2, 128            # tokens, hidden, experts, choices, rows


@pytest.fixture
def lib(monkeypatch):
    r = Recorder()
    monkeypatch.setattr(binding, "_lib", r)
    monkeypatch.setattr(binding, "_raw_stream", lambda: 0)
    monkeypatch.setattr(binding, "_current_device", lambda: 0)
    return r


def i32(*shape, **k):
    return zeros(*shape, dtype=torch.int32, **k)


def with_defaults(f, **defaults):
    def call(**k):
        named = {n: k.pop(n) if n in k else make() for n, make in defaults.items()}
        return f(**named, **k)
    return call


x, g = (lambda: zeros(M, H)), (lambda: zeros(H))
CALLS = {
    "rms": with_defaults(binding.rmsnorm, x=x, gamma=g),
    "rmsq": with_defaults(binding.rmsnorm_quantize, x=x, gamma=g),
    "rms_bwd": with_defaults(binding.rmsnorm_backward, dy=x, z=x, gamma=g, rsigma=lambda: f32(M)),
    "route": with_defaults(binding.route, logits=lambda: zeros(M, E), k=lambda: K),
    "route_bwd": with_defaults(binding.route_backward, dweight=lambda: f32(M, K), logits=lambda: zeros(M, E),
                               index=lambda: i32(M, K)),
    "sort": with_defaults(binding.moe_sort, index=lambda: i32(M, K), experts=lambda: E),
    "dispatch": with_defaults(binding.moe_dispatch, x=x, row=lambda: i32(M, K)),
    "combine": with_defaults(binding.moe_combine, y=lambda: zeros(R, H), row=lambda: i32(M, K)),
    "combine_bwd": with_defaults(binding.moe_combine_backward, dout=x, y=lambda: zeros(R, H), row=lambda: i32(M, K),
                                 weight=lambda: f32(M, K)),
}
OPERANDS = {
    "rms": [dict(x=x()), dict(gamma=g()), dict(residual=x()), dict(out={"y": x()}), dict(residual=x(), out={"z": x()}),
            dict(out={"rsigma": f32(M)}), dict(gamma=f32(H))],
    "rmsq": [dict(x=x()), dict(gamma=g()), dict(residual=x()), dict(residual=x(), out={"z": x()}), dict(dense=True, out={"y": x()}),
             dict(out={"q_row": u8(M, H), "s_row": u8(M, 16)}), dict(colwise=True, out={"q_col": u8(H, M), "s_col": u8(H, 16)}),
             dict(out={"rsigma": f32(M)})],
    "rms_bwd": [dict(dy=x()), dict(z=x()), dict(gamma=g()), dict(rsigma=f32(M)), dict(dz=x()), dict(out={"dx": x()}),
                dict(out={"dgamma": g()}), dict(workspace=u8(1 << 16))],
    "route": [dict(logits=f32(M, E)), dict(bias=f32(E)), dict(out={"index": i32(M, K), "weight": f32(M, K)})],
    "route_bwd": [dict(dweight=f32(M, K)), dict(logits=zeros(M, E)), dict(index=i32(M, K)), dict(out=zeros(M, E))],
    "sort": [dict(index=i32(M, K)), dict(out={"group_m": i32(E)}), dict(out={"row": i32(M, K)}), dict(out={"slot": i32(M * K)})],
    "dispatch": [dict(x=x()), dict(row=i32(M, K)), dict(out=zeros(R, H)), dict(x=u8(M, H), scales=u8(M, 16)),
                 dict(x=u8(M, H), scales=u8(M, 16), out=(u8(R, H), u8(R, 16)))],
    "combine": [dict(y=zeros(R, H)), dict(row=i32(M, K)), dict(weight=f32(M, K)), dict(residual=x()), dict(out=x())],
    "combine_bwd": [dict(dout=x()), dict(y=zeros(R, H)), dict(row=i32(M, K)), dict(weight=f32(M, K)), dict(out={"dy": zeros(R, H)}),
                    dict(out={"dweight": f32(M, K)})],
}
fp16 = torch.float16
WRONG = {
    "rms": [dict(gamma=zeros(H + 1)), dict(residual=zeros(M, H, dtype=fp16)), dict(residual=zeros(M, H + 1)), dict(out={"z": x()}),
            dict(out={"y": zeros(M, 2 * H)}), dict(out={"y": zeros(H, M).t()}), dict(out={"rsigma": zeros(M)}), dict(out={"rsigma": f32(2 * M)[::2]})],
    "rmsq": [dict(x=zeros(M, H, dtype=fp16), gamma=zeros(H, dtype=fp16)), dict(out={"q_row": u8(M, 2 * H)[:, :H], "s_row": u8(M, 16)}),
             dict(out={"q_row": u8(M, H), "s_row": u8(M, 16)[:, :3]}), dict(colwise=True, out={"q_col": u8(M, H), "s_col": u8(H, 16)}),
             dict(out={"z": x()}), dict(rowwise=False, out={"q_row": u8(M, H)}), dict(rowwise=False, out={"s_col": u8(H, 16)}),
             dict(out={"rsigma": f32(M, 1)})],
    "rms_bwd": [dict(dy=zeros(M, H, dtype=fp16)), dict(dz=zeros(M, H + 1)), dict(rsigma=zeros(M)), dict(rsigma=f32(M + 1)),
                dict(out={"dx": zeros(M, H, dtype=fp16)}), dict(out={"dgamma": f32(H)}), dict(workspace=f32(1 << 14))],
    "route": [dict(bias=zeros(E)), dict(bias=f32(E + 1)), dict(out={"index": zeros(M, K, dtype=torch.int64)}),
              dict(out={"weight": f32(M, K + 1)}), dict(out={"weight": f32(M, 2 * K)[:, ::2]})],
    "route_bwd": [dict(dweight=f32(M, K + 1)), dict(index=zeros(M, K, dtype=torch.int64)), dict(dweight=zeros(M, K)),
                  dict(out=f32(M, E)), dict(logits=zeros(M + 1, E))],
    "sort": [dict(index=zeros(M, K, dtype=torch.int64)), dict(index=i32(M, 2 * K)[:, ::2]), dict(out={"row": i32(M * K)}),
             dict(out={"group_m": i32(E + 1)}), dict(out={"slot": i32(M, K)})],
    "dispatch": [dict(row=zeros(M, K, dtype=torch.int64)), dict(row=i32(M + 1, K)), dict(out=zeros(R, H + 1)), dict(out=f32(R, H)),
                 dict(scales=u8(M, 16)), dict(x=u8(M, H), scales=u8(M, 3)), dict(x=u8(M, H), scales=u8(M, 16), out=(u8(R, H), u8(R, 3))),
                 dict(x=u8(M, H + 16), scales=u8(M, 16)), dict(total_rows=R + 1, out=zeros(R, H)), dict(x=zeros(H, M).t())],
    "combine": [dict(weight=zeros(M, K)), dict(weight=f32(M, K + 1)), dict(residual=zeros(M, H + 1)), dict(residual=f32(M, H)), dict(out=f32(M, H)),
                dict(out=zeros(M + 1, H))],
    "combine_bwd": [dict(weight=None), dict(weight=zeros(M, K)), dict(dout=f32(M, H)), dict(dout=zeros(M + 1, H)), dict(out={"dy": x()}),
                    dict(out={"dweight": zeros(M, K)})],
}


@pytest.mark.parametrize("op", sorted(CALLS))
def test_right_operands_reach_the_library(op, lib):
    CALLS[op]()
    for kw in OPERANDS[op]:
        CALLS[op](**kw)
    assert len(lib.launched) == 1 + len(OPERANDS[op])


@pytest.mark.parametrize("op,i", [(op, i) for op in sorted(OPERANDS) for i in range(len(OPERANDS[op]))])
def test_operands_on_another_device_are_refused(op, i, lib):
    for kw in each_moved(OPERANDS[op][i]):
        with pytest.raises(AssertionError):
            CALLS[op](**kw)
        assert not lib.launched


@pytest.mark.parametrize("op", sorted(CALLS))
def test_a_current_device_that_is_another_is_refused(op, lib, monkeypatch):
    monkeypatch.setattr(binding, "_current_device", lambda: 1)
    with pytest.raises(AssertionError):
        CALLS[op]()
    assert not lib.launched


@pytest.mark.parametrize("op,i", [(op, i) for op in sorted(WRONG) for i in range(len(WRONG[op]))])
def test_wrong_shapes_types_and_layouts_are_refused(op, i, lib):
    with pytest.raises(AssertionError):
        CALLS[op](**WRONG[op][i])
    assert not lib.launched


def test_names_that_do_not_exist(lib):
    with pytest.raises(KeyError):
        CALLS["route"](scoring="none")
    with pytest.raises(TypeError):
        CALLS["combine"](y=zeros(R, H, dtype=torch.float64))
    assert not lib.launched


def test_what_comes_back(lib):
    assert set(CALLS["rms"]()) == {"y", "rsigma"} and set(CALLS["rms"](stats=False)) == {"y"}
    assert set(CALLS["rms"](residual=x())) == {"y", "z", "rsigma"}
    assert set(CALLS["rmsq"](rowwise=False, colwise=True, dense=True)) == {"q_col", "s_col", "y", "rsigma"}
    assert set(CALLS["rms_bwd"](dparams=False)) == {"dx"} and set(CALLS["combine_bwd"](dweight=False)) == {"dy"}
    assert CALLS["dispatch"](total_rows=200).shape == (200, H)
    q, s = CALLS["dispatch"](x=u8(M, H), scales=u8(M, 16))
    assert q.shape == (M * K, H) and s.shape == (M * K, 16)
    assert isinstance(x(), Cuda)

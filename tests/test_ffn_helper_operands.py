"""What the LayerNorm and gated helpers refuse before they call the library, on
the CPU: stand-ins that say they are on a CUDA device take the tensors' places
and a recorder the library's, so a call that would hand it a CPU tensor's address
is seen, and nothing runs."""
import pytest
import torch

from mxfp8_block_scaled_quantize_gb300 import binding

M, H, K, F = 40, 64, 128, 32


class Cuda(torch.Tensor):
    """A CPU tensor that says it is on CUDA device 0 (allocations "beside" it stay on the CPU)."""
    is_cuda = property(lambda self: True)

    def get_device(self):
        return 0


class OtherCuda(Cuda):
    def get_device(self):
        return 1


class Recorder:
    """Stands in for the library: notes the launches."""
    def __init__(self):
        self.launched = []

    def __getattr__(self, name):
        def call(*args):
            if name.endswith("_size"):
                return 1024
            self.launched.append(name)
            return 0
        return call


@pytest.fixture
def lib(monkeypatch):
    r = Recorder()
    monkeypatch.setattr(binding, "_lib", r)
    monkeypatch.setattr(binding, "_raw_stream", lambda: 0)
    return r


def zeros(*shape, dtype=torch.bfloat16, kind=Cuda):
    return torch.zeros(shape, dtype=dtype).as_subclass(kind)


def u8(*shape, **k):
    return zeros(*shape, dtype=torch.uint8, **k)


def f32(*shape, **k):
    return zeros(*shape, dtype=torch.float32, **k)


def moved(t):
    """The same tensor on the CPU, and on another device."""
    return [t.as_subclass(torch.Tensor), t.as_subclass(OtherCuda)]


CALLS = {
    "ln": lambda x=None, g=None, b=None, **k: binding.layernorm(zeros(M, H) if x is None else x, zeros(H) if g is None else g, b, **k),
    "ln_bwd": lambda dy=None, x=None, g=None, mu=None, rs=None, **k: binding.layernorm_backward(
        zeros(M, H) if dy is None else dy, zeros(M, H) if x is None else x, zeros(H) if g is None else g,
        f32(M) if mu is None else mu, f32(M) if rs is None else rs, **k),
    "gated": lambda q=None, s=None, w=None, sw=None, **k: binding.gated_gemm(
        u8(M, K) if q is None else q, u8(M, 16) if s is None else s, u8(2 * F, K) if w is None else w,
        u8(2 * F, 16) if sw is None else sw, **k),
    "moe": lambda m=None, q=None, s=None, w=None, sw=None, **k: binding.grouped_gated_gemm(
        zeros(2, dtype=torch.int32) if m is None else m, u8(M, K) if q is None else q, u8(M, 16) if s is None else s,
        u8(2, 2 * F, K) if w is None else w, u8(4 * F, 16) if sw is None else sw, **k),
    "gated_bwd": lambda dh=None, gu=None, **k: binding.gated_backward(
        zeros(M, F) if dh is None else dh, zeros(M, 2 * F) if gu is None else gu, **k),
}

# the operands and outputs of each helper, by keyword
OPERANDS = {
    "ln": [dict(x=zeros(M, H)), dict(g=zeros(H)), dict(b=zeros(H)), dict(out={"y": zeros(M, H)}),
           dict(out={"mu": f32(M), "rsigma": f32(M)})],
    "ln_bwd": [dict(dy=zeros(M, H)), dict(x=zeros(M, H)), dict(g=zeros(H)), dict(mu=f32(M)), dict(rs=f32(M)),
               dict(out={"dx": zeros(M, H)}), dict(out={"dgamma": zeros(H), "dbeta": zeros(H)}), dict(workspace=u8(1 << 16))],
    "gated": [dict(q=u8(M, K)), dict(s=u8(M, 16)), dict(w=u8(2 * F, K)), dict(sw=u8(2 * F, 16)), dict(bias=zeros(2 * F)),
              dict(out=(zeros(M, F), zeros(M, 2 * F)))],
    "moe": [dict(m=zeros(2, dtype=torch.int32)), dict(q=u8(M, K)), dict(s=u8(M, 16)), dict(w=u8(2, 2 * F, K)),
            dict(sw=u8(4 * F, 16)), dict(bias=zeros(2, 2 * F)), dict(out=(zeros(M, F), zeros(M, 2 * F)))],
    "gated_bwd": [dict(dh=zeros(M, F)), dict(gu=zeros(M, 2 * F)), dict(dense=True, out={"d_gate_up": zeros(M, 2 * F)}),
                  dict(out={"q_row": u8(M, 2 * F), "s_row": u8(M, 16)}), dict(out={"q_col": u8(2 * F, 128), "s_col": u8(2 * F, 16)})],
}


def each_moved(kw):
    """kw with one of its tensors on the CPU or on another device, for every one of them."""
    for key, v in kw.items():
        if isinstance(v, torch.Tensor):
            yield from ({**kw, key: t} for t in moved(v))
        elif isinstance(v, dict):
            for name in v:
                yield from ({**kw, key: {**v, name: t}} for t in moved(v[name]))
        elif isinstance(v, tuple):
            for i in range(len(v)):
                yield from ({**kw, key: v[:i] + (t,) + v[i + 1:]} for t in moved(v[i]))


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


# tensors that are too narrow for the call inside wider buffers, whose pitches
# alone would do, and outputs of another type with the right size of element
NARROW = {
    "gated": [dict(s=u8(M, 16)[:, :3]), dict(sw=u8(2 * F, 16)[:, :3])],
    "moe": [dict(s=u8(M, 16)[:, :3]), dict(sw=u8(4 * F, 16)[:, :3])],
    "gated_bwd": [dict(out={"q_row": u8(M, 2 * F), "s_row": u8(M, 16)[:, :1]}),
                  dict(out={"q_col": u8(2 * F, 128)[:, :112], "s_col": u8(2 * F, 16)}),
                  dict(out={"q_col": u8(2 * F, 128), "s_col": u8(2 * F, 16)[:, :3]}),
                  dict(dense=True, out={"d_gate_up": zeros(M, 2 * F, dtype=torch.float16)}),
                  dict(dense=True, out={"d_gate_up": zeros(M, 4 * F)[:, :F]}),
                  dict(out={"q_row": u8(M, 4 * F)[:, :2 * F], "s_row": u8(M, 16)})],
}
WIDE = {
    "gated": [dict(s=u8(M, 32)[:, :4]), dict(sw=u8(2 * F, 48)[:, :16])],
    "moe": [dict(s=u8(M, 32)[:, :5])],
    "gated_bwd": [dict(out={"q_row": u8(M, 2 * F), "s_row": u8(M, 32)[:, :2]}),
                  dict(out={"q_col": u8(2 * F, 160), "s_col": u8(2 * F, 16)[:, :4]}),
                  dict(dense=True, out={"d_gate_up": zeros(M, 4 * F)[:, :2 * F]})],
}


@pytest.mark.parametrize("op,i", [(op, i) for op in sorted(NARROW) for i in range(len(NARROW[op]))])
def test_views_narrower_than_the_call_are_refused(op, i, lib):
    with pytest.raises(AssertionError):
        CALLS[op](**NARROW[op][i])
    assert not lib.launched


@pytest.mark.parametrize("op,i", [(op, i) for op in sorted(WIDE) for i in range(len(WIDE[op]))])
def test_views_of_the_call_s_width_are_taken(op, i, lib):
    CALLS[op](**WIDE[op][i])
    assert len(lib.launched) == 1


# outputs that the library writes in pairs, one of them given
LONE = {
    "ln": [({"mu": f32(M)}, "stats"), ({"rsigma": f32(M)}, "stats")],
    "ln_bwd": [({"dbeta": zeros(H)}, "dparams")],
    "gated_bwd": [({"q_row": u8(M, 2 * F)}, "rowwise"), ({"s_row": u8(M, 16)}, "rowwise"),
                  ({"q_col": u8(2 * F, 128)}, "colwise"), ({"s_col": u8(2 * F, 16)}, "colwise")],
}
PAIRS = {"stats": ("mu", "rsigma"), "dparams": ("dgamma", "dbeta"), "rowwise": ("q_row", "s_row"), "colwise": ("q_col", "s_col")}


@pytest.mark.parametrize("op,i", [(op, i) for op in sorted(LONE) for i in range(len(LONE[op]))])
def test_a_lone_output_is_kept_beside_a_new_one_or_refused(op, i, lib):
    out, switch = LONE[op][i]
    o = CALLS[op](out=out)
    (name, t), = out.items()
    assert o[name] is t and all(k in o for k in PAIRS[switch]) and len(lib.launched) == 1
    with pytest.raises(AssertionError):
        CALLS[op](out=out, **{switch: False})
    assert len(lib.launched) == 1


def test_a_given_dgamma_does_not_take_the_place_of_dbeta(lib):
    g = zeros(H)
    o = CALLS["ln_bwd"](out={"dgamma": g})
    assert o["dgamma"] is g and o["dbeta"].shape == g.shape
    o = CALLS["ln_bwd"](out={"dgamma": g}, dparams=False)      # (asked for by giving it; dbeta was not)
    assert o["dgamma"] is g and "dbeta" not in o

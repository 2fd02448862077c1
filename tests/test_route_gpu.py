"""GPU parity of te_mx_route and te_mx_route_backward against the float64 oracle:
choices exactly, weights and gradients within derived bounds; ties, masked experts,
rows that a mask leaves empty, NaN and infinities, the type's lowest value, every
scoring, odd numbers of experts, pitches, one token to many, graphs and streams; the
gradients also against differences."""
import numpy as np
import pytest
import torch

from mxfp8_block_scaled_quantize_gb300 import binding
from oracle import moe_oracle as M
from tests.test_layernorm_gpu import T, assert_within, check_untouched, f64, guarded

pytestmark = pytest.mark.gpu

HOW = [dict(scoring=s, renormalise=r) for s in ("softmax", "sigmoid") for r in (True, False)]


def make(tokens, experts, t, seed, pad=0):
    g = torch.Generator().manual_seed(seed)
    view, _ = guarded(tokens, experts, experts + pad, T[t])
    view.copy_((2 * torch.randn(tokens, experts, generator=g)).to(T[t]))
    return view, (0.5 * torch.randn(experts, generator=g)).cuda(), g


def check(logits, k, t, bias=None, scoring="softmax", renormalise=True, scale=1.0, dweight=None, pad=0):
    tokens, experts = logits.shape
    index, ibuf = guarded(tokens, k, k, torch.int32)
    weight, wbuf = guarded(tokens, k, k, torch.float32)
    how = dict(scoring=scoring, renormalise=renormalise, scale=scale)
    binding.route(logits, k, bias=bias, out={"index": index, "weight": weight}, **how)
    binding.te_mx_device_status()
    check_untouched(index, ibuf)
    check_untouched(weight, wbuf)
    l = logits.float().cpu().numpy()
    want = M.route_index(l, k, None if bias is None else bias.cpu().numpy())
    assert np.array_equal(index.cpu().numpy(), want), "choices"
    w, b = M.route_weights(l, want, scoring, renormalise, scale), M.route_weights_bound(l, want, scoring, renormalise, scale)
    assert_within(f64(weight), w, b, "weights")
    if dweight is not None:
        d, dbuf = guarded(tokens, experts, experts + pad, T[t])
        binding.route_backward(dweight, logits, index, out=d, **how)
        binding.te_mx_device_status()
        check_untouched(d, dbuf)
        g = dweight.cpu().numpy()
        assert_within(f64(d), M.route_backward(g, l, want, scoring, renormalise, scale),
                      M.route_backward_bound(g, l, want, scoring, renormalise, scale, t), "dlogits")
    return index, weight


@pytest.mark.parametrize("tokens,experts,k", [(1, 1, 1), (1, 8, 2), (7, 33, 5), (100, 64, 6), (33, 60, 4), (257, 128, 8), (40, 160, 6),
                                              (65, 256, 8), (19, 300, 32), (9, 1024, 32), (5, 1000, 7), (3, 32, 32), (2000, 96, 3)])
@pytest.mark.parametrize("t", ["bf16", "fp16", "fp32"])
def test_routes(tokens, experts, k, t):
    for i, how in enumerate(HOW):
        logits, bias, g = make(tokens, experts, t, tokens + experts + i, pad=(0, 3)[i % 2])
        dw = torch.randn(tokens, k, generator=g).cuda()
        check(logits, k, t, bias=bias if i % 2 else None, scale=(1.0, 2.5)[i // 2], dweight=dw, pad=i, **how)
        check(logits, k, t, bias=None if i % 2 else bias, dweight=dw, **how)


@pytest.mark.parametrize("how", HOW)
def test_ties_masks_and_rows_that_a_mask_leaves_empty(how):
    inf, low = float("inf"), torch.finfo(torch.float32).min
    l = torch.zeros(8, 40)
    l[1, ::3] = 1.0                                   # ties in a higher class
    l[2, 5:] = -inf                                   # five experts left, seven wanted
    l[3, :] = -inf                                    # none left
    l[4, :] = low                                     # masks of the type's lowest value
    l[4, 7] = 0.0
    l[5, :] = low
    l[6, ::2] = -0.0                                  # equal to 0
    l[7, 3:] = -inf
    l = l.cuda()
    dw = torch.arange(56, device="cuda", dtype=torch.float32).view(8, 7) / 56
    index, weight = check(l, 7, "fp32", dweight=dw, **how)
    assert index[3].tolist() == list(range(7)) and index[5].tolist() == list(range(7)) and index[0].tolist() == list(range(7))
    assert index[2].tolist() == list(range(7)) and torch.all(weight[2, 5:] == 0) and torch.all(weight[3] == 0)
    d = binding.route_backward(dw, l, index, **how)
    assert torch.isfinite(d).all() and torch.all(d[3] == 0) and torch.all(d[2, 5:] == 0)


@pytest.mark.parametrize("how", HOW)
def test_nan_and_infinite_logits(how):
    l = torch.randn(6, 64, generator=torch.Generator().manual_seed(1))
    clean = binding.route(l.cuda(), 4, **how)
    l[1, 3], l[2, :], l[4, 9] = float("nan"), float("nan"), float("inf")
    o = binding.route(l.cuda(), 4, **how)
    assert np.array_equal(o["index"].cpu().numpy(), M.route_index(l.numpy(), 4))
    assert o["index"][2].tolist() == [0, 1, 2, 3] and o["index"][4, 0] == 9 and torch.isnan(o["weight"][2]).all()
    keep = [0, 3, 5]
    assert torch.equal(o["weight"][keep], clean["weight"][keep]) and torch.equal(o["index"][keep], clean["index"][keep])
    d = binding.route_backward(torch.ones(6, 4, device="cuda"), l.cuda(), o["index"], **how)
    assert torch.isfinite(d[keep]).all()


def test_a_bias_that_chooses_experts_of_vanishing_score():
    l = torch.zeros(3, 16).cuda()
    l[:, 0] = 500.0
    bias = torch.zeros(16, device="cuda")
    bias[4:8] = 1000.0
    index, weight = check(l, 4, "fp32", bias=bias, dweight=torch.rand(3, 4).cuda())
    assert index[0].tolist() == [4, 5, 6, 7] and torch.all(weight == 0.25)
    check(l, 4, "fp32", bias=bias, renormalise=False, dweight=torch.rand(3, 4).cuda())


@pytest.mark.parametrize("how", HOW)
def test_dropped_choices_take_no_part_in_the_gradient(how):
    logits, _, g = make(30, 48, "fp32", 5)
    index = binding.route(logits, 6, **how)["index"]
    index[::3, 2], index[5], index[7, 0] = -1, -1, 48
    dw = torch.randn(30, 6, generator=g).cuda()
    d = binding.route_backward(dw, logits, index, scale=1.5, **how)
    l, i, w = logits.cpu().numpy(), index.cpu().numpy(), dw.cpu().numpy()
    assert_within(f64(d), M.route_backward(w, l, i, scale=1.5, **how), M.route_backward_bound(w, l, i, scale=1.5, t="fp32", **how), "dlogits")
    assert torch.all(d[5] == 0)


@pytest.mark.parametrize("how", HOW)
def test_gradient_against_differences(how):
    logits, _, g = make(4, 20, "fp32", 9)
    o = binding.route(logits, 5, scale=2.0, **how)
    dw = torch.randn(4, 5, generator=g)
    d = f64(binding.route_backward(dw.cuda(), logits, o["index"], scale=2.0, **how))
    l, i = f64(logits), o["index"].cpu().numpy()
    loss = lambda v: (M.route_weights(v, i, scale=2.0, **how) * dw.double().numpy()).sum()  # noqa: E731
    for seed in range(3):
        v = np.random.default_rng(seed).standard_normal(l.shape)
        diff = (loss(l + 1e-5 * v) - loss(l - 1e-5 * v)) / 2e-5
        assert abs((d * v).sum() - diff) < 1e-6 + 300 * 2.0 ** -24 * np.abs(d * v).sum()


def test_repeats_in_a_graph_and_on_a_stream_and_takes_no_tokens():
    logits, bias, g = make(300, 128, "bf16", 3)
    dw = torch.randn(300, 8, generator=g).cuda()

    def step(**k):
        o = binding.route(logits, 8, bias=bias, **k)
        return o["index"], o["weight"], binding.route_backward(dw, logits, o["index"], **k)

    want = step()
    torch.cuda.synchronize()
    got = [step(stream=torch.cuda.Stream())]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got.append(step())
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for r in got for a, b in zip(want, r))
    o = binding.route(logits[:0], 8)
    assert o["index"].shape == (0, 8) and binding.route_backward(dw[:0], logits[:0], o["index"]).shape == (0, 128)

"""The float64 oracle of the RMSNorm, router, sorting and combine operators
against torch autograd in float64, brute force and hand-made cases (no GPU)."""
import numpy as np
import pytest
import torch

from oracle import moe_oracle as M


def rng(seed):
    return np.random.default_rng(seed)


def test_rmsnorm_and_its_gradient_against_autograd():
    g = rng(0)
    z, dy, dz, ga = g.standard_normal((5, 40)), g.standard_normal((5, 40)), g.standard_normal((5, 40)), g.standard_normal(40)
    zt, gt = (torch.tensor(v, requires_grad=True) for v in (z, ga))
    y = zt * torch.rsqrt((zt * zt).mean(1, keepdim=True) + 1e-5) * gt
    (y * torch.tensor(dy)).sum().backward()
    want, rs = M.rmsnorm(z, ga)
    dx, dga = M.rmsnorm_backward(dy, z, ga, rs, dz)
    assert np.allclose(want, y.detach().numpy(), rtol=1e-13)
    assert np.allclose(dx, zt.grad.numpy() + dz, rtol=1e-11, atol=1e-13) and np.allclose(dga, gt.grad.numpy(), rtol=1e-11)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalise", [True, False])
def test_router_and_its_gradient_against_autograd(scoring, renormalise):
    g = rng(1)
    l, dw = g.standard_normal((6, 20)), g.standard_normal((6, 4))
    index = M.route_index(l, 4)
    lt = torch.tensor(l, requires_grad=True)
    p = torch.softmax(lt, 1) if scoring == "softmax" else torch.sigmoid(lt)
    c = p.gather(1, torch.tensor(index, dtype=torch.int64))
    w = 2.5 * (c / c.sum(1, keepdim=True) if renormalise else c)
    (w * torch.tensor(dw)).sum().backward()
    assert np.allclose(M.route_weights(l, index, scoring, renormalise, 2.5), w.detach().numpy(), rtol=1e-12)
    assert np.allclose(M.route_backward(dw, l, index, scoring, renormalise, 2.5), lt.grad.numpy(), rtol=1e-9, atol=1e-13)


def test_choices_with_ties_nan_infinities_and_a_bias():
    inf, nan = np.inf, np.nan
    l = np.array([[1, 3, 3, 2], [-inf, -inf, -inf, -inf], [nan, 1, nan, -inf], [0.0, -0.0, inf, 0.0]], np.float32)
    assert M.route_index(l, 4).tolist() == [[1, 2, 3, 0], [0, 1, 2, 3], [1, 3, 0, 2], [2, 0, 1, 3]]
    assert M.route_index(l[:1], 2, np.array([5, 0, 0, 0], np.float32)).tolist() == [[0, 1]]
    w = M.route_weights(l[1:2], np.array([[0, 1]]), "softmax", True, 1.0)
    assert np.array_equal(w, [[0, 0]])


def test_sort_by_hand_and_round_trip():
    group_m, row, slot = M.moe_sort(np.array([[2, 0], [-1, 2], [0, 7]], np.int32), 3)
    assert group_m.tolist() == [2, 0, 2] and row.tolist() == [[2, 0], [-1, 3], [1, -1]] and slot.tolist() == [1, 4, 0, 3, -1, -1]
    g = rng(2)
    index = g.integers(-1, 9, (50, 3)).astype(np.int32)
    group_m, row, slot = M.moe_sort(index, 8)
    kept = int(group_m.sum())
    assert np.array_equal(row.reshape(-1)[slot[:kept]], np.arange(kept)) and np.all(slot[kept:] == -1)
    assert np.all(np.diff(index.reshape(-1)[slot[:kept]]) >= 0)


def test_combine_and_its_gradient_against_autograd():
    g = rng(3)
    row = np.array([[2, 0], [-1, 1], [-1, -1]], np.int32)
    y, w, res, dout = g.standard_normal((4, 5)), g.standard_normal((3, 2)), g.standard_normal((3, 5)), g.standard_normal((3, 5))
    yt, wt = (torch.tensor(v, requires_grad=True) for v in (y, w))
    out = torch.tensor(res) + torch.stack([wt[0, 0] * yt[2] + wt[0, 1] * yt[0], wt[1, 1] * yt[1], 0 * yt[0]])
    (out * torch.tensor(dout)).sum().backward()
    assert np.allclose(M.moe_combine(y, row, w, res)[0], out.detach().numpy())
    assert np.allclose(M.moe_dweight(dout, y, row)[0], wt.grad.numpy())


def test_bounds_hold_for_fp32_evaluations_and_are_not_wide():
    g = rng(4)
    z = g.standard_normal((8, 512)).astype(np.float32)
    ga = g.standard_normal(512).astype(np.float32)
    rs = (1 / np.sqrt((z * z).mean(1, dtype=np.float32) + np.float32(1e-5))).astype(np.float32)
    y, want_rs = M.rmsnorm(z, ga)
    got = (z * rs[:, None] * ga).astype(np.float32)
    bound = M.rmsnorm_bound(y, 64, "fp32")
    assert np.all(np.abs(got - y) <= bound) and np.all(bound <= 1e-5 * np.abs(y) + 1e-30)
    l = g.standard_normal((30, 64)).astype(np.float32)
    index = M.route_index(l, 6)
    e = np.exp(l - l.max(1, keepdims=True)).astype(np.float32)
    p = e / e.sum(1, keepdims=True, dtype=np.float32)
    w = np.take_along_axis(p, index.astype(np.int64), 1)
    b = M.route_weights_bound(l, index, "softmax", False, 1.0)
    want = M.route_weights(l, index, "softmax", False, 1.0)
    assert np.all(np.abs(w - want) <= b) and np.all(b <= 2e-5 * want)


@pytest.mark.parametrize("mistake", ["mean for mean square", "eps outside the root", "unweighted", "last of a tie"])
def test_planted_mistakes_are_seen(mistake):
    g = rng(5)
    if mistake in ("mean for mean square", "eps outside the root"):
        z, ga = 0.02 * g.standard_normal((4, 64)) + 0.01, np.ones(64)
        y, _ = M.rmsnorm(z, ga)
        rs = 1 / np.sqrt(z.var(1) + 1e-5) if "mean sq" in mistake else 1 / (np.sqrt((z * z).mean(1)) + 1e-5)
        assert np.any(np.abs(z * rs[:, None] - y) > M.rmsnorm_bound(y, 200, "bf16"))
    elif mistake == "unweighted":
        y, row = g.standard_normal((6, 8)), np.arange(6).reshape(3, 2)
        w = np.full((3, 2), 0.98)
        out, size = M.moe_combine(y, row, w)
        assert np.any(np.abs(M.moe_combine(y, row)[0] - out) > M.moe_combine_bound(out, size, 2, "bf16"))
    else:
        l = np.array([[1, 5, 5, 0]], np.float32)
        assert M.route_index(l, 1)[0, 0] != 3 - np.argmax(l[0, ::-1])

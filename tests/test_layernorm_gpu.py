"""GPU parity of te_mx_layernorm and te_mx_layernorm_backward against the
float64 oracle, within its derived error bounds: every type, rows of one
element to long ones, odd widths, pitches and alignments, single rows and
many, extreme and non-finite rows, in-place use, absent outputs, other
streams, graph capture, determinism, canary-guarded outputs; the gradients
also against differences of the forward definition."""
import numpy as np
import pytest
import torch

from mxfp8_block_scaled_quantize_gb300 import binding
from oracle import ffn_oracle as F

pytestmark = pytest.mark.gpu

T = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
GUARD = 64


def f64(t):
    return t.detach().double().cpu().numpy()


def row_sum_depth(hidden):
    # chain of a row sum: at most ceil(hidden / 256) terms in a thread (fewer
    # threads than that take short rows), five butterfly levels, up to 32 warps
    # and up to 8 blocks of a row
    return -(-hidden // 256) + 64 + 5 + 32 + 8


def column_sum_depth(rows):
    # rows of one partial sum (at least 152 of them, if there are that many
    # rows), 32 row groups of a block, and the partials: 304 / 8 in a warp and 8 warps
    return -(-rows // 152) + 32 + 38 + 8


def guarded(rows, hidden, ld, dtype, offset=0):
    """[rows, hidden] view with pitch ld, `offset` elements into a buffer of
    sentinels; returns (view, whole buffer)."""
    buf = torch.full((offset + rows * ld + GUARD,), 7.0, dtype=dtype, device="cuda")
    return buf[offset:offset + rows * ld].view(rows, ld)[:, :hidden], buf


def check_untouched(view, buf):
    """Nothing but the view's own elements was written."""
    mask = torch.ones_like(buf, dtype=torch.bool)
    mask.as_strided(view.shape, view.stride(), view.storage_offset()).fill_(False)
    assert torch.all(buf[mask] == 7.0), "write outside the output"


def make(rows, hidden, t, tp, seed, pad=0, offset=0, mean=0.5, std=1.0):
    g = torch.Generator().manual_seed(seed)
    v = torch.randn(rows, hidden, generator=g) * std * torch.exp2(2 * torch.rand(rows, 1, generator=g)) \
        + mean * torch.randn(rows, 1, generator=g)
    dy = 0.1 * torch.randn(rows, hidden, generator=g)
    out = []
    for m in (v, dy):
        view, _ = guarded(rows, hidden, hidden + pad, T[t], offset)
        view.copy_(m.to(T[t]))
        out.append(view)
    ga = (1 + 0.1 * torch.randn(hidden, generator=g)).to(T[tp]).cuda()
    be = (0.1 * torch.randn(hidden, generator=g)).to(T[tp]).cuda()
    return out[0], out[1], ga, be


def assert_within(got, want, bound, what):
    bad = ~(np.abs(got - want) <= bound)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} outside the bound; first {i}: got {got[i]!r} "
                             f"want {want[i]!r} bound {bound[i]!r}")


def check_forward(x, ga, be, t, pad=0, offset=0, eps=1e-5):
    rows, hidden = x.shape
    y, ybuf = guarded(rows, hidden, hidden + pad, T[t], offset)
    mu, mbuf = guarded(1, rows, rows, torch.float32)
    rs, rbuf = guarded(1, rows, rows, torch.float32)
    binding.layernorm(x, ga, be, eps=eps, out={"y": y, "mu": mu[0], "rsigma": rs[0]})
    binding.te_mx_device_status()
    for v, b in ((y, ybuf), (mu, mbuf), (rs, rbuf)):
        check_untouched(v, b)
    xv, gv, bv = f64(x), f64(ga), None if be is None else f64(be)
    depth = row_sum_depth(hidden)
    want, wmu, wrs = F.layernorm(xv, gv, bv, eps)
    dmu, rho = F.layernorm_stat_bounds(xv, eps, depth)
    assert_within(f64(mu)[0], wmu, dmu + 2.0 ** -149, "mu")
    assert_within(f64(rs)[0], wrs, rho * wrs, "rsigma")
    assert_within(f64(y), want, F.layernorm_bound(xv, gv, 0.0 if be is None else bv, eps, depth, t), "y")
    return mu[0].clone(), rs[0].clone(), y


def check_backward(dy, x, ga, mu, rs, t, tp, pad=0, offset=0):
    rows, hidden = x.shape
    dx, xbuf = guarded(rows, hidden, hidden + pad, T[t], offset)
    dga, gbuf = guarded(1, hidden, hidden, T[tp])
    dbe, bbuf = guarded(1, hidden, hidden, T[tp])
    need = binding.te_mx_layernorm_backward_workspace_size(rows, hidden)
    ws = torch.full((need + 256,), 0xFF, dtype=torch.uint8, device="cuda")      # NaN bits on entry
    binding.layernorm_backward(dy, x, ga, mu, rs, out={"dx": dx, "dgamma": dga[0], "dbeta": dbe[0]}, workspace=ws[:need])
    binding.te_mx_device_status()
    for v, b in ((dx, xbuf), (dga, gbuf), (dbe, bbuf)):
        check_untouched(v, b)
    assert torch.all(ws[need:] == 0xFF), "write past the workspace"
    args = [f64(v) for v in (dy, x, ga, mu, rs)]
    want = F.layernorm_backward(*args)
    bounds = F.layernorm_backward_bounds(*args, row_sum_depth(hidden), column_sum_depth(rows), t, tp)
    for got, w, b, name in zip((f64(dx), f64(dga)[0], f64(dbe)[0]), want, bounds, ("dx", "dgamma", "dbeta")):
        assert_within(got, w, b, name)
    return dx, dga[0], dbe[0]


SHAPES = [(1, 1), (1, 7168), (2, 3), (3, 64), (5, 1023), (130, 1000), (37, 256), (700, 520), (300, 1024), (9, 2056),
          (160, 4096), (64, 7168), (3, 8192), (5, 8200), (19, 16384), (2, 32768), (2, 40000), (1, 70000)]


@pytest.mark.parametrize("rows,hidden", SHAPES)
@pytest.mark.parametrize("t,tp", [("bf16", "bf16"), ("fp16", "fp32"), ("fp32", "fp32")])
def test_forward_and_backward(rows, hidden, t, tp):
    x, dy, ga, be = make(rows, hidden, t, tp, rows * 7 + hidden)
    mu, rs, _ = check_forward(x, ga, be, t)
    check_backward(dy, x, ga, mu, rs, t, tp)


@pytest.mark.parametrize("t,tp", [("bf16", "fp32"), ("fp16", "fp16")])
@pytest.mark.parametrize("pad,offset", [(8, 0), (1, 0), (0, 1), (3, 5), (24, 8)])
def test_pitches_and_alignments(t, tp, pad, offset):
    for rows, hidden in ((33, 512), (65, 1000)):
        x, dy, ga, be = make(rows, hidden, t, tp, pad * 10 + offset, pad, offset)
        mu, rs, _ = check_forward(x, ga, be, t, pad, offset)
        check_backward(dy, x, ga, mu, rs, t, tp, pad, offset)


def test_mixed_alignment_of_the_operands():
    # x on 16-byte rows, dy and the outputs off them (and the other way round)
    x, _, ga, be = make(40, 768, "bf16", "bf16", 1)
    _, dy, _, _ = make(40, 768, "bf16", "bf16", 2, pad=3, offset=1)
    mu, rs, _ = check_forward(x, ga, be, "bf16", pad=1, offset=3)
    check_backward(dy, x, ga, mu, rs, "bf16", "bf16", pad=8, offset=0)
    check_backward(x, dy, ga, mu, rs, "bf16", "bf16", pad=5, offset=0)
    g4 = torch.ones(768 + 1, dtype=torch.bfloat16, device="cuda")[1:]            # gamma off 4-byte boundaries
    check_forward(x, g4, be, "bf16")
    check_backward(dy, x, g4, mu, rs, "bf16", "bf16")


@pytest.mark.parametrize("rows,hidden,t", [(4100, 1024, "bf16"), (8192, 512, "fp16"), (2500, 64, "fp32"), (1000, 7168, "bf16"),
                                           (700, 16384, "fp32")])
def test_many_rows(rows, hidden, t):
    x, dy, ga, be = make(rows, hidden, t, t, rows + hidden)
    mu, rs, _ = check_forward(x, ga, be, t)
    check_backward(dy, x, ga, mu, rs, t, t)


def test_without_shift_statistics_or_gradients():
    x, dy, ga, _ = make(50, 640, "bf16", "bf16", 4)
    mu, rs, y = check_forward(x, ga, None, "bf16")
    o = binding.layernorm(x, ga, None, stats=False)
    assert set(o) == {"y"} and torch.equal(o["y"], y)
    dx, dga, dbe = check_backward(dy, x, ga, mu, rs, "bf16", "bf16")
    o = binding.layernorm_backward(dy, x, ga, mu, rs, dparams=False)
    assert set(o) == {"dx"} and torch.equal(o["dx"], dx)
    ws = torch.empty(binding.te_mx_layernorm_backward_workspace_size(50, 640), dtype=torch.uint8, device="cuda")
    g2 = torch.empty_like(ga)
    stream = torch.cuda.current_stream().cuda_stream
    binding.te_mx_layernorm_backward(dy.data_ptr(), 640, x.data_ptr(), 640, 50, 640, binding.BF16, ga.data_ptr(),
                                     binding.BF16, mu.data_ptr(), rs.data_ptr(), 0, 0, g2.data_ptr(), 0, ws.data_ptr(),
                                     ws.numel(), stream)                          # dgamma alone
    assert torch.equal(g2, dga)


@pytest.mark.parametrize("hidden", [1000, 1001])
def test_in_place(hidden):
    x, dy, ga, be = make(77, hidden, "bf16", "bf16", 5)
    mu, rs, y = check_forward(x, ga, be, "bf16")
    dx, dga, dbe = check_backward(dy, x, ga, mu, rs, "bf16", "bf16")
    d = dy.clone()
    o = binding.layernorm_backward(d, x, ga, mu, rs, out={"dx": d})
    assert torch.equal(o["dx"], dx) and torch.equal(o["dgamma"], dga) and torch.equal(o["dbeta"], dbe)
    v = x.clone()
    binding.layernorm(v, ga, be, out={"y": v})
    assert torch.equal(v, y)


def test_no_rows():
    ga = torch.ones(96, device="cuda")
    x = torch.empty(0, 96, device="cuda")
    o = binding.layernorm(x, ga, ga)
    assert o["y"].shape == (0, 96)
    g = {"dgamma": torch.full((96,), 3.0, device="cuda"), "dbeta": torch.full((96,), 3.0, device="cuda")}
    e = torch.empty(0, device="cuda")
    o = binding.layernorm_backward(x, x, ga, e, e, out=g)
    assert torch.all(o["dgamma"] == 0) and torch.all(o["dbeta"] == 0)


def test_constant_large_mean_and_tiny_rows():
    g = torch.Generator().manual_seed(1)
    x = torch.randn(64, 2048, generator=g).cuda()
    x[0] = 2.5                                        # variance 0: y = beta
    x[1] = 1e4 + x[1]                                 # |mean| >> deviation
    x[2] *= 1e-6                                      # variance far below epsilon
    x[3] *= 1e15
    x[4] = 0
    ga, be = torch.rand(2048, generator=g).cuda(), torch.rand(2048, generator=g).cuda()
    mu, rs, y = check_forward(x, ga, be, "fp32")
    assert torch.equal(y[0], be) and torch.equal(y[4], be)
    dy = torch.randn(64, 2048, generator=g).cuda()
    check_backward(dy, x, ga, mu, rs, "fp32", "fp32")


@pytest.mark.parametrize("hidden", [512, 515])
def test_non_finite_rows_stay_in_their_rows(hidden):
    x, dy, ga, be = make(40, hidden, "bf16", "bf16", 8)
    clean = binding.layernorm(x, ga, be)
    bad = x.clone()
    bad[3, 100], bad[9, 0], bad[30, hidden - 1] = float("nan"), float("inf"), -float("inf")
    got = binding.layernorm(bad, ga, be)
    rows = torch.tensor([3, 9, 30], device="cuda")
    assert torch.isnan(got["y"][rows].float()).all() and torch.isnan(got["rsigma"][rows]).all()
    keep = torch.ones(40, dtype=torch.bool, device="cuda")
    keep[rows] = False
    assert torch.equal(got["y"][keep], clean["y"][keep]) and torch.equal(got["mu"][keep], clean["mu"][keep])
    o = binding.layernorm_backward(dy, bad, ga, got["mu"], got["rsigma"])
    w = binding.layernorm_backward(dy, x, ga, clean["mu"], clean["rsigma"])
    assert torch.isnan(o["dx"][rows].float()).all() and torch.equal(o["dx"][keep], w["dx"][keep])
    assert torch.isnan(o["dgamma"].float()).all() and torch.equal(o["dbeta"], w["dbeta"])


def test_backward_of_the_quantising_layernorm():
    x, dy, ga, be = make(128, 1024, "bf16", "bf16", 9)
    q = binding.layernorm_quantize(x, ga, be)
    check_backward(dy, x, ga, q["mu"], q["rsigma"], "bf16", "bf16")


def test_dx_against_differences():
    # directional derivatives of sum(dy y) by the float64 forward definition
    x, dy, ga, be = make(6, 200, "fp32", "fp32", 10)
    o = binding.layernorm(x, ga, be)
    dx = f64(binding.layernorm_backward(dy, x, ga, o["mu"], o["rsigma"])["dx"])
    xv, dv, gv, bv = f64(x), f64(dy), f64(ga), f64(be)
    loss = lambda t: (dv * F.layernorm(t, gv, bv)[0]).sum()  # noqa: E731
    for seed in range(3):
        v = np.random.default_rng(seed).standard_normal(xv.shape)
        h = 1e-5
        diff = (loss(xv + h * v) - loss(xv - h * v)) / (2 * h)
        # fp32 gradients: |dx| u times a chain of a few hundred operations
        assert abs((dx * v).sum() - diff) < 1e-6 + 300 * 2.0 ** -24 * np.abs(dx * v).sum()


def test_deterministic_on_another_stream_and_in_a_graph():
    x, dy, ga, be = make(600, 2048, "bf16", "bf16", 11)
    a = binding.layernorm(x, ga, be)
    b = binding.layernorm_backward(dy, x, ga, a["mu"], a["rsigma"])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        a2 = binding.layernorm(x, ga, be)
        b2 = binding.layernorm_backward(dy, x, ga, a2["mu"], a2["rsigma"])
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a3 = binding.layernorm(x, ga, be)
        b3 = binding.layernorm_backward(dy, x, ga, a3["mu"], a3["rsigma"])
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    for p, q in ((a2, b2), (a3, b3)):
        assert all(torch.equal(a[k], p[k]) for k in a) and all(torch.equal(b[k], q[k]) for k in b)


def test_offsets_past_32_bits():
    # the last rows of a matrix whose elements' offsets pass 2^31 (bytes past 2^32)
    rows, hidden, ld = 2200, 512, 1 << 20
    buf = torch.empty(rows * ld, dtype=torch.bfloat16, device="cuda")
    x = buf.view(rows, ld)[:, :hidden]
    g = torch.Generator().manual_seed(2)
    v = torch.randn(rows, hidden, generator=g).to(torch.bfloat16).cuda()
    ga, be = torch.ones(hidden, dtype=torch.bfloat16, device="cuda"), torch.zeros(hidden, dtype=torch.bfloat16, device="cuda")
    want = binding.layernorm(v, ga, be)
    x.copy_(v)
    got = binding.layernorm(x, ga, be)
    w = binding.layernorm_backward(v, v, ga, want["mu"], want["rsigma"])
    o = binding.layernorm_backward(x, x, ga, got["mu"], got["rsigma"])
    binding.layernorm(x, ga, be, out={"y": x})
    assert torch.equal(got["y"], want["y"]) and torch.equal(x, want["y"])
    assert all(torch.equal(o[k], w[k]) for k in w)

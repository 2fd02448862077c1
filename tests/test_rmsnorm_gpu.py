"""GPU parity of te_mx_rmsnorm, te_mx_rmsnorm_quantize and te_mx_rmsnorm_backward
against the float64 oracle, within its derived error bounds: every type, rows of
one element to long ones, odd widths, pitches and alignments, single rows and many,
extreme and non-finite rows, in-place use, absent operands, other streams, graphs,
canary-guarded outputs; z bit-exact, codes and scales bit-exact given the kernel's
rsigma; the gradients also against differences of the forward definition."""
import numpy as np
import pytest
import torch

from mxfp8_block_scaled_quantize_gb300 import binding
from oracle import moe_oracle as M
from oracle import mx_oracle as O
from tests import _util as U
from tests.test_layernorm_gpu import T, assert_within, check_untouched, f64, guarded

pytestmark = pytest.mark.gpu


def row_depth(hidden):
    # chain of a row's sum: at most ceil(hidden / 256) terms in a thread (long rows: 64 + 64
    # + 8), five butterfly levels, five or up to 32 across the warps
    return -(-hidden // 256) + 160


def column_depth(rows):
    # rows of one partial sum (at least 152 of them, if there are that many rows), the few
    # rows' 10 + 2 + 16, 32 row groups of a block, and the partials: 304 / 32 in a warp and 32 warps
    return -(-rows // 152) + 32 + 32 + 42


def make(rows, hidden, t, tp, seed, pad=0, offset=0, std=1.0):
    """x, residual, dy, dz (views of pitch hidden + pad, `offset` elements into their buffers) and gamma."""
    g = torch.Generator().manual_seed(seed)
    scale = torch.exp2(4 * torch.rand(rows, 1, generator=g) - 2)
    out = []
    for s in (std * scale, std * scale, 0.1, 0.2):
        view, _ = guarded(rows, hidden, hidden + pad, T[t], offset)
        view.copy_((torch.randn(rows, hidden, generator=g) * s).to(T[t]))
        out.append(view)
    return *out, (1 + 0.1 * torch.randn(hidden, generator=g)).to(T[tp]).cuda()


def check_forward(x, res, ga, t, pad=0, offset=0, eps=1e-5):
    rows, hidden = x.shape
    y, ybuf = guarded(rows, hidden, hidden + pad, T[t], offset)
    rs, rbuf = guarded(1, rows, rows, torch.float32)
    out, bufs = {"y": y, "rsigma": rs[0]}, [(y, ybuf), (rs, rbuf)]
    if res is not None:
        out["z"], zbuf = guarded(rows, hidden, hidden + pad, T[t], offset)
        bufs.append((out["z"], zbuf))
    want_z = x.clone() if res is None else (x.float() + res.float()).to(T[t])
    binding.rmsnorm(x, ga, eps=eps, residual=res, out=out)
    binding.te_mx_device_status()
    for v, b in bufs:
        check_untouched(v, b)
    if res is not None:
        assert torch.equal(out["z"], want_z), "z"
    z, d = f64(want_z), row_depth(hidden)
    want, wrs = M.rmsnorm(z, f64(ga), eps)
    assert_within(f64(rs)[0], wrs, M.rmsnorm_rho(d) * wrs, "rsigma")
    assert_within(f64(y), want, M.rmsnorm_bound(want, d, t), "y")
    return want_z, rs[0].clone(), y


def check_backward(dy, z, ga, rs, dz, t, tp, pad=0, offset=0):
    rows, hidden = z.shape
    dx, xbuf = guarded(rows, hidden, hidden + pad, T[t], offset)
    dga, gbuf = guarded(1, hidden, hidden, T[tp])
    need = binding.te_mx_rmsnorm_backward_workspace_size(rows, hidden)
    ws = torch.full((need + 256,), 0xFF, dtype=torch.uint8, device="cuda")      # NaN bits on entry
    binding.rmsnorm_backward(dy, z, ga, rs, dz=dz, out={"dx": dx, "dgamma": dga[0]}, workspace=ws[:need])
    binding.te_mx_device_status()
    for v, b in ((dx, xbuf), (dga, gbuf)):
        check_untouched(v, b)
    assert torch.all(ws[need:] == 0xFF), "write past the workspace"
    args = [f64(v) for v in (dy, z, ga, rs)] + [None if dz is None else f64(dz)]
    bounds = M.rmsnorm_backward_bounds(*args, row_depth(hidden), column_depth(rows), t, tp)
    for got, w, b, name in zip((f64(dx), f64(dga)[0]), M.rmsnorm_backward(*args), bounds, ("dx", "dgamma")):
        assert_within(got, w, b, name)
    return dx, dga[0]


def check_codes(z, rs, ga, out, rowwise, colwise):
    """Codes and scales: exactly the quantisation of fl(fl(z rs) gamma) for the kernel's rs."""
    y = (z.float().cpu() * rs.cpu()[:, None]) * ga.float().cpu()
    for name, axis in (("row", 1), ("col", 0)):
        if not (rowwise if axis == 1 else colwise):
            assert "q_" + name not in out
            continue
        q, s = O.quantize_mx_values(y.double().numpy(), axis)
        n = s.shape[1]
        U.assert_bytes_equal(out["q_" + name].cpu().numpy(), q, name + " codes")
        U.assert_bytes_equal(out["s_" + name][:, :n].cpu().numpy(), s, name + " scales")


def check_quantize(x, res, ga, rowwise=True, colwise=True, dense=True, eps=1e-5):
    rows, hidden = x.shape
    out, bufs = {}, {}
    if rowwise:
        out["q_row"], bufs["q_row"] = U.guarded_u8(rows, hidden)
        out["s_row"], bufs["s_row"] = U.guarded_u8(rows, binding.te_mx_scale_pitch(hidden))
    if colwise:
        out["q_col"], bufs["q_col"] = U.guarded_u8(hidden, rows)
        out["s_col"], bufs["s_col"] = U.guarded_u8(hidden, binding.te_mx_scale_pitch(rows))
    rs, rbuf = guarded(1, rows, rows, torch.float32)
    views = [(rs, rbuf)]
    out["rsigma"] = rs[0]
    for name in (["y"] if dense else []) + (["z"] if res is not None else []):
        out[name], buf = guarded(rows, hidden, hidden + 8, torch.bfloat16, 8)
        views.append((out[name], buf))
    want_z = x.clone() if res is None else (x.float() + res.float()).to(torch.bfloat16)
    binding.rmsnorm_quantize(x, ga, eps=eps, residual=res, rowwise=rowwise, colwise=colwise, dense=dense, out=out)
    binding.te_mx_device_status()
    for v, b in views:
        check_untouched(v, b)
    for n in bufs:
        U.check_guard(bufs[n], out[n].numel())
    for n, blocks in (("s_row", hidden // 32), ("s_col", rows // 32)):
        assert n not in out or torch.all(out[n][:, blocks:] == U.CANARY), "scale padding was written"
    if res is not None:
        assert torch.equal(out["z"], want_z)
    z, d = f64(want_z), row_depth(hidden)
    want, wrs = M.rmsnorm(z, f64(ga), eps)
    assert_within(f64(rs)[0], wrs, M.rmsnorm_rho(d) * wrs, "rsigma")
    if dense:
        assert_within(f64(out["y"]), want, M.rmsnorm_bound(want, d, "bf16"), "y")
    check_codes(want_z, rs[0], ga, out, rowwise, colwise)
    return out


SHAPES = [(1, 1), (1, 7168), (2, 3), (3, 64), (5, 1023), (130, 1000), (37, 256), (700, 520), (300, 1024), (9, 2056),
          (160, 4096), (64, 7168), (3, 8192), (5, 8200), (19, 16384), (2, 32768), (2, 40000), (1, 70000), (3, 16390), (310, 8193)]


@pytest.mark.parametrize("rows,hidden", SHAPES)
@pytest.mark.parametrize("t,tp", [("bf16", "bf16"), ("fp16", "fp32"), ("fp32", "fp32"), ("bf16", "fp32"), ("fp16", "fp16")])
def test_forward_and_backward(rows, hidden, t, tp):
    x, res, dy, dz, ga = make(rows, hidden, t, tp, rows * 7 + hidden)
    z, rs, _ = check_forward(x, res, ga, t)
    check_backward(dy, z, ga, rs, dz, t, tp)
    z, rs, _ = check_forward(x, None, ga, t)
    check_backward(dy, z, ga, rs, None, t, tp)


@pytest.mark.parametrize("t,tp", [("bf16", "fp32"), ("fp16", "fp16")])
@pytest.mark.parametrize("pad,offset", [(8, 0), (1, 0), (0, 1), (3, 5), (24, 8)])
def test_pitches_and_alignments(t, tp, pad, offset):
    for rows, hidden in ((33, 512), (65, 1000), (400, 96)):
        x, res, dy, dz, ga = make(rows, hidden, t, tp, pad * 10 + offset, pad, offset)
        z, rs, _ = check_forward(x, res, ga, t, pad, offset)
        check_backward(dy, z, ga, rs, dz, t, tp, pad, offset)


def test_mixed_alignment_of_the_operands():
    x, res, dy, dz, ga = make(40, 768, "bf16", "bf16", 1)
    ux, ures, udy, udz, _ = make(40, 768, "bf16", "bf16", 2, pad=3, offset=1)
    z, rs, _ = check_forward(x, ures, ga, "bf16")
    check_forward(ux, res, ga, "bf16")
    check_forward(x, res, ga, "bf16", pad=1, offset=3)
    check_backward(udy, z, ga, rs, dz, "bf16", "bf16")
    check_backward(dy, z, ga, rs, udz, "bf16", "bf16")
    check_backward(dy, z, ga, rs, dz, "bf16", "bf16", pad=5)
    g4 = torch.ones(768 + 1, dtype=torch.bfloat16, device="cuda")[1:]            # gamma off 4-byte boundaries
    check_forward(x, res, g4, "bf16")
    check_backward(dy, z, g4, rs, dz, "bf16", "bf16")


@pytest.mark.parametrize("rows,hidden,t", [(4100, 1024, "bf16"), (8192, 512, "fp16"), (2500, 64, "fp32"), (1000, 7168, "bf16"),
                                           (700, 16384, "fp32"), (5000, 24, "bf16"), (3001, 1021, "fp16"), (1111, 8200, "fp32"),
                                           (500, 16384, "bf16"), (600, 14336, "bf16"), (400, 20000, "bf16")])
def test_many_rows(rows, hidden, t):
    x, res, dy, dz, ga = make(rows, hidden, t, t, rows + hidden)
    z, rs, _ = check_forward(x, res, ga, t)
    check_backward(dy, z, ga, rs, dz, t, t)


@pytest.mark.parametrize("rows,hidden", [(32, 32), (1, 64), (5, 4096), (64, 96), (160, 7168), (2048, 544), (3, 32768), (96, 16384),
                                         (416, 8224), (33, 160), (1184, 1024), (64, 32768), (32, 25600), (160, 25632)])
@pytest.mark.parametrize("tp", ["bf16", "fp32"])
def test_quantised(rows, hidden, tp):
    x, res, _, _, ga = make(rows, hidden, "bf16", tp, rows + hidden, pad=8)
    both = rows % 32 == 0
    check_quantize(x, res, ga, colwise=both)
    check_quantize(x, None, ga, colwise=both, dense=False)
    if both:
        check_quantize(x, res, ga, rowwise=False)
        check_quantize(x, None, ga, rowwise=False, dense=False)
    check_quantize(x, res, ga, rowwise=False, colwise=False)


def test_quantised_blocks_of_zeros_non_finite_and_extreme_values():
    x, _, _, _, ga = make(64, 256, "bf16", "bf16", 3)
    x[3] = 0                                          # scale bytes of zero blocks
    x[5, 40], x[9, 0], x[30, 255] = float("nan"), float("inf"), -float("inf")
    x[11] *= 1e-30
    x[13, 32:64] = 0                                  # one block of zeros
    x[14] = 3e38                                      # the sum of squares overflows: rsigma 0
    out = binding.rmsnorm_quantize(x, ga, colwise=True)
    rs = out["rsigma"]
    assert torch.isnan(rs[5]) and rs[9] == 0 and rs[30] == 0 and rs[14] == 0
    check_codes(x, rs, ga, out, True, True)


def test_in_place():
    for hidden in (1000, 1001, 17000, 17001):
        x, res, dy, dz, ga = make(77, hidden, "bf16", "bf16", 5)
        z, rs, y = check_forward(x, res, ga, "bf16")
        dx, dga = check_backward(dy, z, ga, rs, dz, "bf16", "bf16")
        for into in ("x", "residual"):
            v = {"x": x.clone(), "residual": res.clone()}
            o = binding.rmsnorm(v["x"], ga, residual=v["residual"], out={"z": v[into]})
            assert torch.equal(v[into], z) and torch.equal(o["y"], y)
            v = {"x": x.clone(), "residual": res.clone()}
            other = "residual" if into == "x" else "x"
            binding.rmsnorm(v["x"], ga, residual=v["residual"], out={"z": v[into], "y": v[other]})
            assert torch.equal(v[into], z) and torch.equal(v[other], y)
        v = z.clone()
        binding.rmsnorm(v, ga, out={"y": v})
        assert torch.equal(v, y)
        for into in ("dy", "z", "dz"):
            v = {"dy": dy.clone(), "z": z.clone(), "dz": dz.clone()}
            o = binding.rmsnorm_backward(v["dy"], v["z"], ga, rs, dz=v["dz"], out={"dx": v[into]})
            assert torch.equal(o["dx"], dx)
            # (another kernel where dx overlaps, so another order of the sums)
            size = np.abs(f64(dy) * f64(z) * f64(rs)[:, None]).sum(0)
            assert_within(f64(o["dgamma"]), f64(dga), 2.0 ** -7 * np.abs(f64(dga)) + 3 * column_depth(77) * 2.0 ** -24 * size, "dgamma")
    x, res, _, _, ga = make(64, 512, "bf16", "bf16", 6)
    want = binding.rmsnorm_quantize(x, ga, residual=res, colwise=True, dense=True)
    v, r = x.clone(), res.clone()
    got = binding.rmsnorm_quantize(v, ga, residual=r, colwise=True, dense=True, out={"z": r, "y": v})
    assert all(torch.equal(want[k], got[k]) for k in want if k[0] != "s")
    assert torch.equal(want["s_row"][:, :16], got["s_row"][:, :16]) and torch.equal(want["s_col"][:, :2], got["s_col"][:, :2])


def test_columns_of_one_wide_buffer():
    # z and y beside x in rows of one buffer: apart, although their ranges of memory cross
    g = torch.Generator().manual_seed(8)
    buf = torch.randn(50, 3 * 256, generator=g).to(torch.bfloat16).cuda()
    x, z, y = buf[:, :256], buf[:, 256:512], buf[:, 512:]
    res, ga = x.flip(0).clone(), torch.ones(256, dtype=torch.bfloat16, device="cuda")
    want = binding.rmsnorm(x.clone(), ga, residual=res)
    binding.rmsnorm(x, ga, residual=res, out={"z": z, "y": y})
    assert torch.equal(z, want["z"]) and torch.equal(y, want["y"])


def test_no_rows():
    ga = torch.ones(96, device="cuda")
    x = torch.empty(0, 96, device="cuda")
    assert binding.rmsnorm(x, ga, residual=x)["z"].shape == (0, 96)
    e = torch.empty(0, device="cuda")
    o = binding.rmsnorm_backward(x, x, ga, e, out={"dgamma": torch.full((96,), 3.0, device="cuda")})
    assert torch.all(o["dgamma"] == 0) and o["dx"].shape == (0, 96)
    q = binding.rmsnorm_quantize(x.bfloat16(), ga, colwise=True)
    assert q["q_row"].shape == (0, 96)


def test_constant_tiny_and_large_rows():
    g = torch.Generator().manual_seed(1)
    x = torch.randn(64, 2048, generator=g).cuda()
    x[0], x[4] = 2.5, 0
    x[2] *= 1e-6                                      # the mean square is far below epsilon
    x[3] *= 1e15
    ga, dy = torch.rand(2048, generator=g).cuda(), torch.randn(64, 2048, generator=g).cuda()
    z, rs, y = check_forward(x, None, ga, "fp32")
    assert torch.all(y[4] == 0)
    check_backward(dy, z, ga, rs, dy, "fp32", "fp32")


@pytest.mark.parametrize("hidden", [512, 515])
def test_non_finite_rows_stay_in_their_rows(hidden):
    x, res, dy, dz, ga = make(40, hidden, "bf16", "bf16", 8)
    clean = binding.rmsnorm(x, ga, residual=res)
    bad = x.clone()
    bad[3, 100], bad[9, 0] = float("nan"), float("inf")
    got = binding.rmsnorm(bad, ga, residual=res)
    rows = torch.tensor([3, 9], device="cuda")
    keep = torch.ones(40, dtype=torch.bool, device="cuda")
    keep[rows] = False
    assert torch.isnan(got["y"][3].float()).all() and torch.isnan(got["y"][9, 0]) and got["rsigma"][9] == 0
    assert all(torch.equal(got[k][keep], clean[k][keep]) for k in clean)
    o = binding.rmsnorm_backward(dy, got["z"], ga, got["rsigma"], dz=dz)
    w = binding.rmsnorm_backward(dy, clean["z"], ga, clean["rsigma"], dz=dz)
    assert torch.isnan(o["dx"][3].float()).all() and torch.equal(o["dx"][keep], w["dx"][keep])


def test_dx_against_differences():
    x, _, dy, dz, ga = make(6, 200, "fp32", "fp32", 10)
    o = binding.rmsnorm(x, ga)
    b = binding.rmsnorm_backward(dy, x, ga, o["rsigma"], dz=dz)
    xv, dv, gv, zv = f64(x), f64(dy), f64(ga), f64(dz)
    loss = lambda t, g: (dv * M.rmsnorm(t, g)[0]).sum() + (zv * t).sum()  # noqa: E731
    for seed in range(3):
        r = np.random.default_rng(seed)
        v, w = r.standard_normal(xv.shape), r.standard_normal(gv.shape)
        h = 1e-5
        dx, dga = f64(b["dx"]), f64(b["dgamma"])
        # fp32 gradients: |dx| u times a chain of a few hundred operations
        diff = (loss(xv + h * v, gv) - loss(xv - h * v, gv)) / (2 * h)
        assert abs((dx * v).sum() - diff) < 1e-6 + 300 * 2.0 ** -24 * np.abs(dx * v).sum()
        diff = (loss(xv, gv + h * w) - loss(xv, gv - h * w)) / (2 * h)
        assert abs((dga * w).sum() - diff) < 1e-6 + 300 * 2.0 ** -24 * np.abs(dga * w).sum()


def same(a, b):
    return a.keys() == b.keys() and all(torch.equal(a[k], b[k]) for k in a if not k.startswith("s_"))


@pytest.mark.parametrize("rows,hidden", [(608, 2048), (64, 1024), (352, 1001)])
def test_repeats_on_another_stream_and_in_a_graph(rows, hidden):
    x, res, dy, dz, ga = make(rows, hidden, "bf16", "bf16", 11)

    def step():
        a = binding.rmsnorm(x, ga, residual=res)
        q = binding.rmsnorm_quantize(x, ga, residual=res, colwise=True) if hidden % 32 == 0 else a
        return a, q, binding.rmsnorm_backward(dy, a["z"], ga, a["rsigma"], dz=dz)

    want = step()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = [step() for _ in range(3)]
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got.append(step())
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    for g in got:
        assert all(same(p, q) for p, q in zip(want, g))


def test_stream_argument():
    x, res, dy, dz, ga = make(320, 2048, "bf16", "bf16", 12)
    fwd = binding.rmsnorm(x, ga, residual=res)
    calls = [lambda **k: binding.rmsnorm(x, ga, residual=res, **k),
             lambda **k: binding.rmsnorm_quantize(x, ga, residual=res, colwise=True, **k),
             lambda **k: binding.rmsnorm_backward(dy, fwd["z"], ga, fwd["rsigma"], dz=dz, **k)]
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


def test_offsets_past_32_bits():
    # the last rows of a matrix whose elements' offsets pass 2^31 (bytes past 2^32)
    rows, hidden, ld = 2208, 512, 1 << 20
    buf = torch.empty(rows * ld, dtype=torch.bfloat16, device="cuda")
    x = buf.view(rows, ld)[:, :hidden]
    v = torch.randn(rows, hidden, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    ga = torch.ones(hidden, dtype=torch.bfloat16, device="cuda")
    want = binding.rmsnorm(v, ga, residual=v)
    x.copy_(v)
    got = binding.rmsnorm(x, ga, residual=x)
    q, wq = (binding.rmsnorm_quantize(m, ga, colwise=True) for m in (x, v))
    w = binding.rmsnorm_backward(v, v, ga, want["rsigma"], dz=v)
    o = binding.rmsnorm_backward(x, x, ga, got["rsigma"], dz=x)
    binding.rmsnorm(x, ga, residual=x, out={"z": x})
    assert torch.equal(got["y"], want["y"]) and torch.equal(x, want["z"])
    assert same(o, w) and same(q, wq)

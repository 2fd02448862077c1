"""GPU parity of te_mx_gated_backward: the bf16 gradient against the float64
oracle within its derived bound and against differences, the quantised copies
bit for bit against the oracle's quantisation of that bf16 gradient (tokens
zero-padded to 128 in the column-wise copy), and the two gradients that the
GEMMs make of them.  Rows from one to many strips, widths that fill no unit or
strip, pitches, in-place use, each output alone, extreme and NaN inputs,
streams and graphs; canary-guarded outputs."""
import numpy as np
import pytest
import torch

from mxfp8_block_scaled_quantize_gb300 import binding
from oracle import ffn_oracle as F
from oracle import mx_oracle as O
from tests import _util as U

pytestmark = pytest.mark.gpu


def f64(t):
    return t.double().cpu().numpy()


def make(rows, n, seed, scale=1e-3):
    g = torch.Generator().manual_seed(seed)
    dh = (torch.randn(rows, n, generator=g) * scale).to(torch.bfloat16).cuda()
    gu = (torch.randn(rows, 2 * n, generator=g) * 2).to(torch.bfloat16).cuda()
    return dh, gu


def run(dh, gu, kind, dense=True, rowwise=True, colwise=True, ld_extra=0):
    rows, n = dh.shape
    kp = (rows + 127) // 128 * 128
    out, bufs = {}, {}
    if dense:
        out["d_gate_up"], bufs["d_gate_up"] = U.guarded_bf16(rows, 2 * n)
    if rowwise:
        out["q_row"], bufs["q_row"] = U.guarded_u8(rows, 2 * n)
        out["s_row"], bufs["s_row"] = U.guarded_u8(rows, binding.te_mx_scale_pitch(2 * n))
    if colwise:
        w, bufs["q_col"] = U.guarded_u8(2 * n, kp + ld_extra)
        s, bufs["s_col"] = U.guarded_u8(2 * n, binding.te_mx_scale_pitch(kp) + ld_extra)
        out["q_col"], out["s_col"] = w, s
    binding.gated_backward(dh, gu, activation=kind, dense=dense, rowwise=rowwise, colwise=colwise, out=out)
    binding.te_mx_device_status()
    for k, b in bufs.items():
        U.check_guard(b, out[k].numel())
    if rowwise:
        s = out["s_row"].cpu().numpy()
        assert np.all(s[:, 2 * n // 32:] == U.CANARY), "row-wise scale padding was written"
    if colwise:
        q, s = out["q_col"].cpu().numpy(), out["s_col"].cpu().numpy()
        assert np.all(q[:, kp:] == U.CANARY) and np.all(s[:, kp // 32:] == U.CANARY), "column-wise padding was written"
    return out


def check_dense(d, dh, gu, kind):
    n = dh.shape[1]
    h, g, u = f64(dh), f64(gu[:, :n]), f64(gu[:, n:])
    for got, want, bound, name in zip((f64(d[:, :n]), f64(d[:, n:])), F.gated_backward(h, g, u, kind),
                                      F.gated_backward_bounds(h, g, u, kind), ("dg", "du")):
        bad = ~(np.abs(got - want) <= bound)
        if bad.any():
            i = tuple(np.argwhere(bad)[0])
            raise AssertionError(f"{name}: {int(bad.sum())} of {bad.size} outside the bound; first {i}: got {got[i]!r} "
                                 f"want {want[i]!r} bound {bound[i]!r} at g {g[i]!r} u {u[i]!r} dh {h[i]!r}")


def check_codes(out, d):
    """The copies in ``out`` are the oracle's of the bf16 gradient d."""
    rows, n2 = d.shape
    bits = U.bf16_bits(d)
    if "q_row" in out:
        q, s = O.quantize_rowwise(bits)
        U.assert_bytes_equal(out["q_row"].cpu().numpy(), q, "row-wise codes")
        U.assert_bytes_equal(out["s_row"].cpu().numpy()[:, :n2 // 32], s, "row-wise scales")
    if "q_col" in out:
        kp = (rows + 127) // 128 * 128
        padded = np.zeros((kp, n2), np.uint16)
        padded[:rows] = bits
        q, s = O.quantize_colwise(padded)
        U.assert_bytes_equal(out["q_col"].cpu().numpy()[:, :kp], q, "column-wise codes")
        U.assert_bytes_equal(out["s_col"].cpu().numpy()[:, :kp // 32], s, "column-wise scales")


@pytest.mark.parametrize("kind", ["silu", "gelu", "relu"])
@pytest.mark.parametrize("rows,n", [(1, 32), (2, 16), (31, 64), (33, 96), (64, 512), (100, 544), (128, 1024), (130, 4128),
                                    (257, 160), (5, 7168)])
def test_dense_alone(rows, n, kind):
    dh, gu = make(rows, n, rows + n)
    out = run(dh, gu, kind, rowwise=False, colwise=False)
    check_dense(out["d_gate_up"], dh, gu, kind)


@pytest.mark.parametrize("kind", ["silu", "gelu", "relu"])
@pytest.mark.parametrize("rows,n", [(1, 32), (31, 64), (32, 96), (33, 160), (64, 512), (100, 544), (128, 1024), (129, 1056),
                                    (300, 4128), (1000, 768)])
def test_every_output(rows, n, kind):
    dh, gu = make(rows, n, rows * 3 + n)
    out = run(dh, gu, kind)
    check_dense(out["d_gate_up"], dh, gu, kind)
    check_codes(out, out["d_gate_up"])
    alone = run(dh, gu, kind, rowwise=False, colwise=False)
    assert torch.equal(alone["d_gate_up"], out["d_gate_up"])


@pytest.mark.parametrize("dense", [False, True])
@pytest.mark.parametrize("rowwise,colwise", [(True, True), (True, False), (False, True)])
def test_outputs_alone_and_together(dense, rowwise, colwise):
    dh, gu = make(200, 672, 5)
    want = run(dh, gu, "silu", rowwise=False, colwise=False)["d_gate_up"]
    out = run(dh, gu, "silu", dense=dense, rowwise=rowwise, colwise=colwise, ld_extra=32)
    if dense:
        assert torch.equal(out["d_gate_up"], want)
    check_codes(out, want)


def test_several_strips_per_block():
    # more strips (64 rows x 512 columns) than the GPU has SMs, the last of a band cut
    for rows, n in ((64 * 41, 512 * 9 + 96), (64 * 200, 64)):
        dh, gu = make(rows, n, rows)
        d = run(dh, gu, "silu", rowwise=False, colwise=False)["d_gate_up"]
        check_codes(run(dh, gu, "silu", dense=False), d)
        check_dense(d, dh, gu, "silu")


def test_pitches_and_in_place():
    dh0, gu0 = make(70, 96, 6)
    dh, gu = torch.zeros(70, 120, dtype=torch.bfloat16, device="cuda"), torch.zeros(70, 232, dtype=torch.bfloat16, device="cuda")
    dh[:, :96], gu[:, 8:200] = dh0, gu0
    want = run(dh0, gu0, "gelu")
    got = run(dh[:, :96], gu[:, 8:200], "gelu")
    for k in want:
        assert torch.equal(want[k], got[k]), k
    binding.gated_backward(dh[:, :96], gu[:, 8:200], activation="gelu", dense=True, rowwise=False, colwise=False,
                           out={"d_gate_up": gu[:, 8:200]})
    assert torch.equal(gu[:, 8:200], want["d_gate_up"])
    assert torch.all(gu[:, :8] == 0) and torch.all(gu[:, 200:] == 0)


@pytest.mark.parametrize("kind", ["silu", "gelu", "relu"])
def test_extreme_gates(kind):
    g = torch.Generator().manual_seed(7)
    mag = torch.exp2(torch.rand(64, 128, generator=g) * 140 - 70)
    gate = torch.where(torch.rand(64, 128, generator=g) < 0.5, -mag, mag)
    gate[:, :16] = torch.tensor([0.0, -0.0, 1.0, -1.0, -1.2784, -0.7518, 29.9, 30.1, -29.9, -30.1, 88.0, -88.0, -103.0, 127.0,
                                 3e38, -3e38])
    up = torch.randn(64, 128, generator=g)
    dh = torch.randn(64, 128, generator=g).to(torch.bfloat16).cuda()
    gu = torch.cat([gate, up], 1).to(torch.bfloat16).cuda()
    out = run(dh, gu, kind)
    ok = gu[:, :128].float().abs() < 1e30                # (du of the rest overflows bf16 for some dh)
    h, gv, uv = f64(dh), f64(gu[:, :128]), f64(gu[:, 128:])
    (dg, du), (bg, bu) = F.gated_backward(h, gv, uv, kind), F.gated_backward_bounds(h, gv, uv, kind)
    got, m = f64(out["d_gate_up"]), ok.cpu().numpy()
    assert np.all(np.abs(got[:, :128] - dg) <= bg), "dg"
    assert np.all((np.abs(got[:, 128:] - du) <= bu)[m]), "du"
    check_codes(out, out["d_gate_up"])


def test_nan_reaches_its_element_and_its_blocks_only():
    dh, gu = make(96, 128, 8)
    clean = run(dh, gu, "silu")
    dh2, gu2 = dh.clone(), gu.clone()
    dh2[40, 7], gu2[3, 100], gu2[70, 128 + 50] = float("nan"), float("nan"), float("inf")
    out = run(dh2, gu2, "silu")
    bad = torch.zeros(96, 256, dtype=torch.bool)
    bad[40, 7] = bad[40, 128 + 7] = bad[3, 100] = bad[3, 128 + 100] = bad[70, 50] = True
    d = out["d_gate_up"].cpu()
    assert torch.equal(~torch.isfinite(d), bad) and torch.equal(d[~bad], clean["d_gate_up"].cpu()[~bad])
    check_codes(out, out["d_gate_up"])


def test_against_differences():
    # dg and du of sum(dh h) by central differences of the float64 forward function
    dh, gu = make(8, 64, 9, scale=1.0)
    for kind in ("silu", "gelu"):
        d = f64(run(dh, gu, kind, rowwise=False, colwise=False)["d_gate_up"])
        h, g, u = f64(dh), f64(gu[:, :64]), f64(gu[:, 64:])
        e = 1e-5
        dg = h * (F.gated(g + e, u, kind) - F.gated(g - e, u, kind)) / (2 * e)
        du = h * (F.gated(g, u + e, kind) - F.gated(g, u - e, kind)) / (2 * e)
        bg, bu = F.gated_backward_bounds(h, g, u, kind)
        assert np.all(np.abs(d[:, :64] - dg) <= bg + 1e-8) and np.all(np.abs(d[:, 64:] - du) <= bu + 1e-8)


@pytest.mark.parametrize("rows,n,k", [(256, 128, 256), (200, 192, 128), (1, 64, 128)])
def test_gradients_through_the_gemms(rows, n, k):
    # dX = [dg | du] W and dW = [dg | du]^T X from the copies, W's and X's copies by the framework
    dh, gu = make(rows, n, 10, scale=1.0)
    g = torch.Generator().manual_seed(11)
    x = torch.randn(rows, k, generator=g).to(torch.bfloat16).cuda()
    w = (0.05 * torch.randn(2 * n, k, generator=g)).to(torch.bfloat16).cuda()
    qw = binding.quantize(w, rowwise=False, colwise=True)
    kp = (rows + 127) // 128 * 128
    qx = {"q": torch.empty(k, kp, dtype=torch.uint8, device="cuda"),
          "s": torch.empty(k, binding.te_mx_scale_pitch(kp), dtype=torch.uint8, device="cuda")}
    binding.quantize_colwise_grouped(x, torch.tensor([rows], dtype=torch.int32, device="cuda"), out=qx)
    d = binding.gated_backward(dh, gu, activation="silu")
    dx, _ = binding.gemm(d["q_row"], d["s_row"], qw["q_col"], qw["s_col"])
    dw, _ = binding.gemm(d["q_col"], d["s_col"], qx["q"], qx["s"])
    binding.te_mx_device_status()
    cpu = lambda t: t.cpu().numpy()  # noqa: E731
    for got, (qa, sa), (qb, sb), name in ((dx, (d["q_row"], d["s_row"]), (qw["q_col"], qw["s_col"]), "dX"),
                                          (dw, (d["q_col"], d["s_col"]), (qx["q"], qx["s"]), "dW")):
        kk = qa.shape[1] // 32
        ref = O.mx_gemm(cpu(qa), cpu(sa)[:, :kk], cpu(qb), cpu(sb)[:, :kk])
        assert np.all(np.abs(f64(got) - ref["d"]) <= O.gemm_error_bound(ref["d"], ref["sigma"])), name


def test_on_another_stream_and_in_a_graph():
    dh, gu = make(300, 1024, 12)
    a = binding.gated_backward(dh, gu, dense=True)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = binding.gated_backward(dh, gu, dense=True)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c = binding.gated_backward(dh, gu, dense=True)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    for k, v in a.items():
        n = (1024 * 2 // 32) if k == "s_row" else (384 // 32) if k == "s_col" else v.shape[1]
        assert torch.equal(v[:, :n], b[k][:, :n]) and torch.equal(v[:, :n], c[k][:, :n]), k


def test_no_rows():
    e = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    o = binding.gated_backward(e, torch.empty(0, 128, dtype=torch.bfloat16, device="cuda"), dense=True)
    assert o["d_gate_up"].shape == (0, 128) and o["q_col"].shape == (128, 0)

"""GPU parity of te_mx_gated_gemm and te_mx_grouped_gated_gemm against the
float64 oracle: every activation, with and without bias and pre-activations,
one token to several tiles, output widths that fill no tile, few and many
K-steps, empty and ragged experts, extreme and NaN operands, other streams and
graphs.  The pre-activations may be off by 1e-5 sum|a w| before they are
rounded (the GEMM's own bound); h by what that, the activation's evaluation
and the rounding to bf16 allow (oracle.ffn_oracle.gated_bound).  Scale-pitch
padding is 0xFF (an E8M0 NaN), every output has a canary tail."""
import numpy as np
import pytest
import torch

from mxfp8_block_scaled_quantize_gb300 import binding
from oracle import ffn_oracle as F
from oracle import mx_oracle as O
from tests import _util as U

pytestmark = pytest.mark.gpu

ACC = 1e-5


def operand(rows, cols, seed, std=1.0, outliers=False):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g) * std
    if outliers:
        x[:, [3, cols // 2]] *= 64.0
    return O.quantize_rowwise(U.bf16_bits(x.to(torch.bfloat16)))


def upload(q, s):
    """Codes and scales on the device; scale padding = 0xFF."""
    pitch = binding.te_mx_scale_pitch(q.shape[1])
    sp = np.full((q.shape[0], pitch), 0xFF, np.uint8)
    sp[:, : s.shape[1]] = s
    return torch.from_numpy(q).cuda(), torch.from_numpy(sp).cuda()


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def reference(qa, sa, qw, sw, bias=None):
    """(pre, bound on the fp32 pre-activation's error), float64."""
    a, w = O.dequantize(qa, sa), O.dequantize(qw, sw)
    pre, sigma = a @ w.T, np.abs(a) @ np.abs(w).T
    if bias is not None:
        pre, sigma = pre + bias, sigma + np.abs(bias)
    return pre, ACC * sigma


def compare(h, pre, ref, err, kind):
    n = ref.shape[1] // 2
    g, u = ref[:, :n], ref[:, n:]
    bound = F.gated_bound(g, u, err[:, :n], err[:, n:], kind)
    for got, want, b, name in ((h, F.gated(g, u, kind), bound, "h"),
                               (pre, ref, err + F.round_half(np.abs(ref) + err, "bf16"), "pre")):
        if got is None:
            continue
        bad = ~(np.abs(f64(got) - want) <= b)
        if bad.any():
            i = tuple(np.argwhere(bad)[0])
            raise AssertionError(f"{name}: {int(bad.sum())} of {bad.size} outside the bound; first {i}: got "
                                 f"{f64(got)[i]!r} want {want[i]!r} bound {b[i]!r}")


def run(qa, sa, qw, sw, kind, bias=None, aux=True):
    M, n = qa.shape[0], qw.shape[0] // 2
    h, hbuf = U.guarded_bf16(M, n)
    pre, pbuf = U.guarded_bf16(M, 2 * n) if aux else (None, None)
    binding.gated_gemm(qa, sa, qw, sw, activation=kind, bias=bias, out=(h, pre))
    binding.te_mx_device_status()
    U.check_guard(hbuf, M * n)
    if aux:
        U.check_guard(pbuf, M * 2 * n)
    return h, pre


def check(M, n, K, kind, bias, aux, seed, std=0.05):
    qa, sa = operand(M, K, seed, outliers=True)
    qw, sw = operand(2 * n, K, seed + 1, std=std)
    b = torch.randn(2 * n, generator=torch.Generator().manual_seed(seed + 2)).to(torch.bfloat16) if bias else None
    h, pre = run(*upload(qa, sa), *upload(qw, sw), kind, None if b is None else b.cuda(), aux)
    ref, err = reference(qa, sa, qw, sw, None if b is None else f64(b))
    compare(h, pre, ref, err, kind)


@pytest.mark.parametrize("M,n,K,kind,bias,aux", [
    (1, 16, 128, "silu", False, True),
    (1, 1040, 2048, "gelu", True, False),
    (2, 128, 256, "relu", True, True),
    (7, 272, 640, "silu", True, True),
    (8, 528, 1152, "gelu", False, True),
    (16, 64, 384, "silu", True, False),
    (17, 144, 4096, "relu", False, True),
    (32, 1024, 1024, "silu", False, True),
    (33, 48, 512, "gelu", True, True),
    (64, 336, 2176, "silu", True, True),
    (65, 192, 256, "gelu", False, False),
    (100, 2064, 1024, "silu", True, True),
    (128, 128, 128, "relu", True, True),
    (129, 320, 384, "silu", False, True),
    (200, 96, 640, "gelu", True, True),
    (255, 16, 2048, "silu", False, False),
    (256, 128, 128, "silu", True, True),
    (256, 16, 256, "gelu", True, True),
    (300, 208, 2176, "relu", False, True),
    (333, 528, 640, "gelu", True, True),
    (512, 1024, 2048, "silu", False, False),
    (700, 1360, 512, "silu", True, True),
])
def test_dense(M, n, K, kind, bias, aux):
    check(M, n, K, kind, bias, aux, M + n + K)


def test_several_tiles_per_block():
    # more 256-row tiles than the GPU has pairs of blocks, odd K-step counts
    check(1100, 4240, 2176, "silu", True, True, 1)
    check(2048, 2192, 384, "gelu", False, True, 2)


def test_single_block_tiles_several_per_block():
    check(200, 2 * 152 * 128 + 32, 128, "silu", False, True, 3)


@pytest.mark.parametrize("kind", ["silu", "gelu", "relu"])
def test_large_and_small_gates(kind):
    # gates from 2^-40 to 2^50: the exponential overflows, vanishes, or is 1
    for M in (3, 300):
        qa, sa = operand(M, 256, 5)
        qw, sw = operand(64, 256, 6)
        sa = (sa.astype(np.int64) + (np.arange(M) * 7 % 90 - 40)[:, None]).astype(np.uint8)
        h, pre = run(*upload(qa, sa), *upload(qw, sw), kind)
        ref, err = reference(qa, sa, qw, sw)
        compare(h, pre, ref, err, kind)


@pytest.mark.parametrize("M", [4, 300])
@pytest.mark.parametrize("kind", ["silu", "gelu", "relu"])
def test_nan_blocks_reach_their_rows_and_columns_only(M, kind):
    qa, sa = operand(M, 256, 7)
    qw, sw = operand(2 * 48, 256, 8)
    clean, _ = run(*upload(qa, sa), *upload(qw, sw), kind)
    qa2, sa2, qw2, sw2 = qa.copy(), sa.copy(), qw.copy(), sw.copy()
    qa2[2, 32:64], sa2[2, 1] = 0x7F, 0xFF                 # a token
    qw2[5, :32], sw2[5, 0] = 0x7F, 0xFF                   # a gate row
    qw2[48 + 9, :32], sw2[48 + 9, 0] = 0x7F, 0xFF         # an up row
    h, _ = run(*upload(qa2, sa2), *upload(qw2, sw2), kind)
    bad = torch.zeros(M, 48, dtype=torch.bool)
    bad[2], bad[:, 5], bad[:, 9] = True, True, True
    assert torch.equal(torch.isnan(h.cpu()), bad) and torch.equal(h.cpu()[~bad], clean.cpu()[~bad])


def check_grouped(sizes, n, K, kind, bias, aux, seed, total=None):
    G, m = len(sizes), np.array(sizes)
    rows = int(m.sum()) if total is None else total
    qa, sa = operand(rows, K, seed, outliers=True)
    qw, sw = operand(G * 2 * n, K, seed + 1, std=0.05)
    b = torch.randn(G, 2 * n, generator=torch.Generator().manual_seed(seed + 2)).to(torch.bfloat16) if bias else None
    h, hbuf = U.guarded_bf16(rows, n)
    pre, pbuf = U.guarded_bf16(rows, 2 * n) if aux else (None, None)
    canary = hbuf.clone()
    da, dsa = upload(qa, sa)
    dw, dsw = upload(qw, sw)
    binding.grouped_gated_gemm(torch.tensor(m, dtype=torch.int32, device="cuda"), da, dsa, dw.view(G, 2 * n, K), dsw,
                               activation=kind, bias=None if b is None else b.cuda(), out=(h, pre))
    binding.te_mx_device_status()
    U.check_guard(hbuf, rows * n)
    used = int(m.sum())
    assert torch.equal(hbuf[used * n:], canary[used * n:]), "rows past the experts' were written"
    if aux:
        U.check_guard(pbuf, rows * 2 * n)
    r = 0
    for e, k in enumerate(sizes):
        w = slice(e * 2 * n, (e + 1) * 2 * n)
        if k:
            ref, err = reference(qa[r:r + k], sa[r:r + k], qw[w], sw[w], None if b is None else f64(b[e]))
            compare(h[r:r + k], None if pre is None else pre[r:r + k], ref, err, kind)
        r += k


@pytest.mark.parametrize("sizes,n,K,kind,bias,aux,total", [
    ([1], 16, 128, "silu", True, True, None),
    ([0, 5, 0, 0, 3], 48, 256, "gelu", True, True, None),
    ([1, 1, 1, 1, 1, 1, 1], 144, 384, "silu", False, True, 20),
    ([127, 0, 129, 64, 1], 208, 640, "relu", True, True, None),
    ([300, 0, 513, 31, 0, 255, 700, 400], 272, 512, "silu", True, True, None),       # pair tiles
    ([0, 0, 2500, 0], 128, 2048, "gelu", False, False, 2600),
])
def test_grouped(sizes, n, K, kind, bias, aux, total):
    check_grouped(sizes, n, K, kind, bias, aux, sum(sizes) + n, total)


def test_grouped_sizes_above_the_total_are_reported():
    qa, sa = operand(64, 128, 1)
    qw, sw = operand(2 * 32, 128, 2)
    da, dsa = upload(qa, sa)
    dw, dsw = upload(qw, sw)
    for bad in ([65], [-1]):
        binding.grouped_gated_gemm(torch.tensor(bad, dtype=torch.int32, device="cuda"), da, dsa, dw.view(1, 64, 128), dsw)
        with pytest.raises(binding.TemxError, match="INVALID_ARG"):
            binding.te_mx_device_status()
    binding.te_mx_device_status()


@pytest.mark.parametrize("M", [1, 20, 100, 400])
def test_deterministic_on_another_stream_and_in_a_graph(M):
    qa, sa = operand(M, 2048, 3)
    qw, sw = operand(2 * 256, 2048, 4)
    args = (*upload(qa, sa), *upload(qw, sw))
    h, pre = binding.gated_gemm(*args, aux=True)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        h2, pre2 = binding.gated_gemm(*args, aux=True)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h3, pre3 = binding.gated_gemm(*args, aux=True)
        h4, _ = binding.gated_gemm(*args)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(h, h2) and torch.equal(h, h3) and torch.equal(h, h4)
    assert torch.equal(pre, pre2) and torch.equal(pre, pre3)
    binding.te_mx_device_status()


def test_no_tokens():
    w = torch.zeros(64, 128, dtype=torch.uint8, device="cuda")
    s = torch.zeros(64, 16, dtype=torch.uint8, device="cuda")
    h, pre = binding.gated_gemm(w[:0], s[:0], w, s, aux=True)
    assert h.shape == (0, 32) and pre.shape == (0, 64)

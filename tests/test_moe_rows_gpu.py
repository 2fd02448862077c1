"""GPU parity of te_mx_moe_sort, te_mx_moe_dispatch, te_mx_moe_combine and
te_mx_moe_combine_backward against the oracle: rows exactly, sums within derived
bounds; empty experts, one expert for all, padding tokens, tokens without a row, one
slot to a million, every type and alignment, rows that nothing owns left as they
were, rows out of range reported, in-place use, graphs and streams; and all of them
in a row around the grouped GEMMs."""
import numpy as np
import pytest
import torch

from mxfp8_block_scaled_quantize_gb300 import binding
from oracle import moe_oracle as M
from tests.test_layernorm_gpu import T, assert_within, check_untouched, f64, guarded

pytestmark = pytest.mark.gpu


def choices(tokens, k, experts, seed, kind="even"):
    g = torch.Generator().manual_seed(seed)
    if kind == "one":
        return torch.full((tokens, k), experts - 1, dtype=torch.int32)
    p = torch.ones(experts) if kind == "even" else torch.arange(1, experts + 1).float() ** -1.5
    if kind == "holes" and experts > 4:
        p[::3] = 0
    index = torch.multinomial(p, tokens * k, replacement=True, generator=g).view(tokens, k).to(torch.int32)
    if kind == "padding":
        index[tokens - tokens // 5:] = -1
    if kind == "dropped":
        index[torch.rand(tokens, k, generator=g) < 0.3] = -7
    return index


def check_sort(index, experts):
    n = index.numel()
    gm, gbuf = guarded(1, experts, experts, torch.int32)
    row, rbuf = guarded(1, n, n, torch.int32)
    slot, sbuf = guarded(1, n, n, torch.int32)
    out = {"group_m": gm[0], "row": row.view(index.shape), "slot": slot[0]}
    binding.moe_sort(index.cuda(), experts, out=out)
    for v, b in ((gm, gbuf), (row, rbuf), (slot, sbuf)):
        check_untouched(v, b)
    for got, want, name in zip((out["group_m"], out["row"], out["slot"]), M.moe_sort(index.numpy(), experts), ("group_m", "row", "slot")):
        assert np.array_equal(got.cpu().numpy(), want), name
    return out


@pytest.mark.parametrize("tokens,k,experts", [(1, 1, 1), (1, 8, 8), (31, 1, 5), (33, 2, 1024), (100, 4, 64), (1000, 3, 7), (8192, 1, 16),
                                              (2049, 4, 128), (8193, 8, 128), (16384, 8, 128), (5000, 32, 1000), (131072, 8, 256)])
def test_sort(tokens, k, experts):
    for i, kind in enumerate(("even", "skewed", "holes", "one", "padding", "dropped")):
        if tokens > 20000 and i not in (1, 5):
            continue
        check_sort(choices(tokens, k, experts, tokens + i, kind), experts)
        binding.te_mx_device_status()


def test_sort_of_nothing_and_of_dropped_slots_alone():
    o = binding.moe_sort(torch.empty(0, 4, dtype=torch.int32, device="cuda"), 9)
    assert torch.all(o["group_m"] == 0) and o["slot"].numel() == 0
    check_sort(torch.full((3000, 4), -1, dtype=torch.int32), 9)


def test_an_expert_out_of_range_is_reported_and_has_no_row():
    index = choices(50, 3, 8, 1)
    index[7, 1] = 8
    check_sort(index, 8)
    with pytest.raises(binding.TemxError, match="INVALID_ARG"):
        binding.te_mx_device_status()
    binding.te_mx_device_status()


def rows_of(tokens, k, experts, seed, kind):
    row = M.moe_sort(choices(tokens, k, experts, seed, kind).numpy(), experts)[1]
    return torch.from_numpy(row).cuda(), int((row >= 0).sum())


def matrix(rows, hidden, t, seed, pad=0, offset=0):
    view, _ = guarded(rows, hidden, hidden + pad, T[t], offset)
    view.copy_(torch.randn(rows, hidden, generator=torch.Generator().manual_seed(seed)).to(T[t]))
    return view


@pytest.mark.parametrize("tokens,k,hidden", [(1, 1, 1), (1, 8, 7168), (5, 2, 33), (100, 4, 2048), (333, 6, 1000), (2000, 2, 100), (64, 32, 256), (7, 3, 20001)])
@pytest.mark.parametrize("t", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("pad,offset", [(0, 0), (8, 0), (1, 3)])
def test_dispatch_and_combine(tokens, k, hidden, t, pad, offset):
    kind = ("even", "padding", "dropped")[(tokens + pad) % 3]
    row, kept = rows_of(tokens, k, 16, tokens + hidden, kind)
    r, m = row.cpu().numpy(), tokens * k
    x = matrix(tokens, hidden, t, 1, pad, offset)
    out, buf = guarded(m, hidden, hidden + pad, T[t], offset)
    binding.moe_dispatch(x, row, out=out)
    check_untouched(out, buf)
    want = torch.full_like(out, 7.0)
    live = torch.from_numpy(r >= 0).cuda()
    want[row[live].long()] = x[live.nonzero()[:, 0]]
    assert torch.equal(out, want)                       # rows that no slot has are left alone
    y, res, dout = matrix(m, hidden, t, 2, pad, offset), matrix(tokens, hidden, t, 3), matrix(tokens, hidden, t, 4, pad, offset)
    y[kept:] = float("nan")                             # rows behind the last
    weight = torch.rand(tokens, k, generator=torch.Generator().manual_seed(5)).cuda() - 0.2
    weight[~live] = float("nan")                        # masked places
    yv, wv = f64(y), f64(weight)
    for w, add in ((weight, res), (weight, None), (None, None), (None, res)):
        o, obuf = guarded(tokens, hidden, hidden + pad, T[t], offset)
        binding.moe_combine(y, row, weight=w, residual=add, out=o)
        check_untouched(o, obuf)
        exact, size = M.moe_combine(yv, r, None if w is None else wv, None if add is None else f64(add))
        assert_within(f64(o), exact, M.moe_combine_bound(exact, size, k, t), "combine")
    dy, ybuf = guarded(m, hidden, hidden + pad, T[t], offset)
    dw, wbuf = guarded(tokens, k, k, torch.float32)
    binding.moe_combine_backward(dout, y, row, weight, out={"dy": dy, "dweight": dw})
    check_untouched(dy, ybuf)
    check_untouched(dw, wbuf)
    want = torch.full_like(dy, 7.0)
    want[row[live].long()] = (dout.float()[live.nonzero()[:, 0]] * weight[live][:, None]).to(T[t])
    assert torch.equal(dy, want)
    exact, size = M.moe_dweight(f64(dout), yv, r)
    assert_within(f64(dw), exact, M.moe_dweight_bound(size, hidden), "dweight")
    assert torch.all(dw[~live] == 0)
    binding.te_mx_device_status()


@pytest.mark.parametrize("cols", [32, 128, 2048, 7168])
def test_quantised_rows_with_their_scales(cols):
    tokens, k = 77, 5
    row, kept = rows_of(tokens, k, 12, cols, "dropped")
    g = torch.Generator().manual_seed(1)
    q = torch.randint(0, 256, (tokens, cols), dtype=torch.uint8, generator=g).cuda()
    pitch = binding.te_mx_scale_pitch(cols)
    s = torch.randint(0, 256, (tokens, pitch), dtype=torch.uint8, generator=g).cuda()
    oq, os = (torch.full((tokens * k + 3, n), 0xA5, dtype=torch.uint8, device="cuda") for n in (cols, pitch + 16))
    binding.moe_dispatch(q, row, scales=s, out=(oq, os))
    binding.te_mx_device_status()
    live = row >= 0
    at, token = row[live].long(), live.nonzero()[:, 0]
    wq, ws = torch.full_like(oq, 0xA5), torch.full_like(os, 0xA5)
    wq[at] = q[token]
    ws[at, :cols // 32] = s[token, :cols // 32]
    assert torch.equal(oq, wq) and torch.equal(os, ws)


def test_rows_out_of_range_are_skipped_and_reported():
    x, y = matrix(4, 64, "bf16", 1), matrix(8, 64, "bf16", 2)
    row = torch.tensor([[0, 8], [1, 2], [100, 3], [4, 2 ** 31 - 1]], dtype=torch.int32, device="cuda")
    weight = torch.ones(4, 2, device="cuda")
    skipped = torch.where(row >= 8, -1, row)
    calls = [lambda r: binding.moe_dispatch(x, r, out=torch.zeros(8, 64, dtype=torch.bfloat16, device="cuda")),
             lambda r: binding.moe_combine(y, r, weight=weight),
             lambda r: binding.moe_combine_backward(x, y, r, weight, out={"dy": torch.zeros_like(y)})]
    for f in calls:
        want = f(skipped)
        binding.te_mx_device_status()
        got = f(row)
        with pytest.raises(binding.TemxError, match="INVALID_ARG"):
            binding.te_mx_device_status()
        assert all(torch.equal(got[n], want[n]) for n in want) if isinstance(want, dict) else torch.equal(got, want)


def test_in_place():
    row, _ = rows_of(90, 4, 8, 1, "dropped")
    y, res, dout = matrix(360, 520, "bf16", 1), matrix(90, 520, "bf16", 2), matrix(90, 520, "bf16", 3)
    weight = torch.rand(90, 4).cuda()
    want = binding.moe_combine(y, row, weight=weight, residual=res)
    v = res.clone()
    binding.moe_combine(y, row, weight=weight, residual=v, out=v)
    assert torch.equal(v, want)
    b = binding.moe_combine_backward(dout, y, row, weight, out={"dy": y.clone()})
    v = y.clone()
    o = binding.moe_combine_backward(dout, v, row, weight, out={"dy": v})
    assert torch.equal(o["dy"], b["dy"]) and torch.equal(o["dweight"], b["dweight"])
    assert set(binding.moe_combine_backward(dout, y, row, weight, dweight=False)) == {"dy"}


def test_offsets_past_32_bits():
    hidden, ld, rows = 64, 1 << 20, 2200                     # elements' offsets pass 2^31
    buf = torch.empty(rows * ld, dtype=torch.bfloat16, device="cuda").view(rows, ld)[:, :hidden]
    row = torch.arange(rows, dtype=torch.int32, device="cuda").flip(0).contiguous().view(rows // 2, 2)
    x, weight = matrix(rows // 2, hidden, "bf16", 1), torch.rand(rows // 2, 2).cuda()
    binding.moe_dispatch(x, row, out=buf)
    dense = binding.moe_dispatch(x, row)
    assert torch.equal(buf, dense)
    assert torch.equal(binding.moe_combine(buf, row, weight=weight), binding.moe_combine(dense, row, weight=weight))
    want = binding.moe_combine_backward(x, dense, row, weight)
    got = binding.moe_combine_backward(x, buf, row, weight, out={"dy": buf})
    assert torch.equal(buf, want["dy"]) and torch.equal(got["dweight"], want["dweight"])


@pytest.mark.parametrize("tokens", [40, 4000])
def test_repeats_in_a_graph_and_on_a_stream(tokens):
    index = choices(tokens, 6, 64, 3, "skewed").cuda()
    x, weight = matrix(tokens, 256, "bf16", 1), torch.rand(tokens, 6).cuda()

    def step(**k):
        s = binding.moe_sort(index, 64, **k)
        d = binding.moe_dispatch(x, s["row"], **k)
        b = binding.moe_combine_backward(x, d, s["row"], weight, **k)
        return s["group_m"], s["row"], s["slot"], d, binding.moe_combine(d, s["row"], weight=weight, **k), b["dy"], b["dweight"]

    want = step()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = []
    for _ in range(4):
        got.append(step(stream=s))
        for n in (1 << 12, 1 << 20, 5 << 20):          # what the current stream takes meanwhile
            torch.empty(n, dtype=torch.uint8, device="cuda").fill_(0xFF)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got.append(step())
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for r in got for a, b in zip(want, r))


def test_calls_on_two_streams_at_once():
    # the whole way there and back, on two streams that overlap, each with inputs of its own
    def step(seed, **kw):
        index = choices(9000, 4, 96, seed, "skewed").cuda()
        x, weight = matrix(9000, 512, "bf16", seed), torch.rand(9000, 4, generator=torch.Generator().manual_seed(seed)).cuda()
        ga = torch.ones(512, dtype=torch.bfloat16, device="cuda")

        def run():
            s = binding.moe_sort(index, 96)
            n = binding.rmsnorm_quantize(x, ga, residual=x, dense=True)
            d = binding.moe_dispatch(n["y"], s["row"])
            b = binding.moe_combine_backward(x, d, s["row"], weight)
            g = binding.rmsnorm_backward(binding.moe_combine(b["dy"], s["row"]), n["z"], ga, n["rsigma"], dz=x)
            return s["row"], s["slot"], d, b["dweight"], g["dx"], g["dgamma"]
        return run

    runs = [step(1), step(2)]
    want = [f() for f in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(6):
        for i in (0, 1):
            with torch.cuda.stream(streams[i]):
                got[i].append(runs[i]())
    torch.cuda.synchronize()
    for i in (0, 1):
        assert all(torch.equal(a, b) for r in got[i] for a, b in zip(want[i], r))


def test_gradient_of_dispatch_is_a_combine_without_weights():
    row, kept = rows_of(50, 3, 8, 4, "dropped")
    x, d = matrix(50, 96, "fp32", 1), matrix(150, 96, "fp32", 2)
    out = binding.moe_dispatch(x, row, out=torch.zeros(150, 96, device="cuda"))
    dx = binding.moe_combine(d, row)
    # <dispatch(x), d> = <x, dx>: two sums of 14400 products (u 2^-24 a rounding, chains of up to 150 and more in 64 bits here)
    a, b = (f64(out)[:kept] * f64(d)[:kept]).sum(), (f64(x) * f64(dx)).sum()
    assert abs(a - b) < 4 * 2.0 ** -24 * np.abs(f64(out) * f64(d)).sum()


def test_around_the_grouped_gemms():
    # norm, router, sort, dispatch of the quantised rows, experts, combine: against float64 on the
    # values that the codes stand for
    from oracle import mx_oracle as O
    tokens, hidden, ffn, experts, k = 200, 256, 128, 8, 2
    g = torch.Generator().manual_seed(6)
    randn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x, res = (randn(tokens, hidden).to(torch.bfloat16).cuda() for _ in range(2))
    gamma, w_router = (1 + 0.1 * randn(hidden)).to(torch.bfloat16).cuda(), randn(experts, hidden).cuda() * 0.06
    w_in = (randn(experts * 2 * ffn, hidden) * 0.06).to(torch.bfloat16).cuda()
    w_out = (randn(experts * hidden, ffn) * 0.09).to(torch.bfloat16).cuda()
    qi, qo = binding.quantize(w_in), binding.quantize(w_out)
    n = binding.rmsnorm_quantize(x, gamma, residual=res, dense=True)
    o = binding.route((n["y"].float() @ w_router.t()).contiguous(), k)
    s = binding.moe_sort(o["index"], experts)
    q, sc = binding.moe_dispatch(n["q_row"], s["row"], scales=n["s_row"])
    h, _ = binding.grouped_gated_gemm(s["group_m"], q, sc, qi["q_row"].view(experts, 2 * ffn, hidden), qi["s_row"])
    qh = binding.quantize(h)
    y, _ = binding.grouped_gemm(s["group_m"], qh["q_row"], qh["s_row"], qo["q_row"].view(experts, hidden, ffn), qo["s_row"])
    out = binding.moe_combine(y, s["row"], weight=o["weight"], residual=n["z"])
    binding.te_mx_device_status()
    deq = lambda q, s: O.dequantize(q.cpu().numpy(), s.cpu().numpy()[:, :q.shape[1] // 32])  # noqa: E731
    xv, wi, wo = deq(n["q_row"], n["s_row"]), deq(qi["q_row"], qi["s_row"]), deq(qo["q_row"], qo["s_row"])
    hv = deq(qh["q_row"], qh["s_row"])
    row, slot, index, weight = s["row"].cpu().numpy(), s["slot"].cpu().numpy(), o["index"].cpu().numpy(), f64(o["weight"])
    want = f64(n["z"])
    size = np.abs(want)
    for t in range(tokens):
        for j in range(k):
            e, r = index[t, j], row[t, j]
            assert slot[r] == t * k + j
            gu = wi[e * 2 * ffn:(e + 1) * 2 * ffn] @ xv[t]
            hid = gu[:ffn] / (1 + np.exp(-gu[:ffn])) * gu[ffn:]
            # h is rounded to bf16 (2^-8), then to E4M3 (2^-4 of the block's largest power of two at most)
            assert np.abs(hv[r] - hid).max() <= (2.0 ** -4 + 2.0 ** -7) * np.abs(hid).max() * 2
            v = weight[t, j] * (wo[e * hidden:(e + 1) * hidden] @ hv[r])
            want[t] += v
            size[t] += np.abs(v) + 1e-5 * weight[t, j] * (np.abs(wo[e * hidden:(e + 1) * hidden]) @ np.abs(hv[r]))
    # each expert's row is rounded to bf16 once, the sum once
    assert np.all(np.abs(f64(out) - want) <= 2.0 ** -7 * size + 1e-3 * 2.0 ** -7)


def test_no_rows_at_all():
    # every choice dropped: the experts' rows are empty
    row = torch.full((5, 3), -1, dtype=torch.int32, device="cuda")
    y, weight = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), torch.ones(5, 3, device="cuda")
    x = matrix(5, 64, "bf16", 1)
    assert binding.moe_dispatch(x, row, total_rows=0).shape == (0, 64)
    assert torch.equal(binding.moe_combine(y, row, weight=weight, residual=x), x)
    assert torch.all(binding.moe_combine(y, row) == 0)
    for dweight in (False, True):
        o = binding.moe_combine_backward(x, y, row, weight, dweight=dweight)
        assert o["dy"].shape == (0, 64) and torch.all(o["dweight"] == 0) if dweight else "dweight" not in o
    binding.te_mx_device_status()


@pytest.mark.parametrize("k", [1, 5])
@pytest.mark.parametrize("hidden", [1 << 24, (1 << 24) - 1])
def test_the_longest_rows(k, hidden):
    # one choice of each token has a row, so the sum is that row
    y = torch.randn(3, hidden, device="cuda")
    row = torch.full((2, k), -1, dtype=torch.int32, device="cuda")
    row[0, k // 2], row[1, 0] = 2, 1
    out = binding.moe_combine(y, row)
    assert torch.equal(out[0], y[2]) and torch.equal(out[1], y[1])
    binding.te_mx_device_status()

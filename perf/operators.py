"""Cases for the LayerNorm and gated feed-forward operators: inputs, a plain
form in elementary torch operations, and the framework's calls.

Operators (a row is a token):

* LayerNorm forward: mu, var over the row (biased), rsigma = 1/sqrt(var + eps),
  y = (x - mu) rsigma gamma + beta.
* LayerNorm backward: dx, dgamma, dbeta from dy, x, mu and rsigma.
* Gated feed-forward, forward: [g | u] = deq(X) deq(W)^T (+ bias) on MXFP8
  operands (E4M3 codes, one E8M0 scale per 32), W = [W_gate; W_up], h =
  act(g) u in bf16, and for training [g | u] in bf16.  Dense, and grouped over
  the experts of a mixture.
* Gated feed-forward, backward: dg = dh u act'(g), du = dh act(g), each rounded
  once to bf16; as they are, or MXFP8-quantised both ways (row-wise, and
  column-wise with the tokens zero-padded to a multiple of 128) and multiplied:
  dX = [dg | du] W, dW = [dg | du]^T X.
"""
import math

import torch

own = False

EPS = 1e-5
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token through a serving step: launch and call latency
        dict(name="ln_token", op="ln_fwd", rows=1, hidden=7168, dtype="bf16", params="bf16", pad=0, stats=False),
        # a training step of the large dense FFN: 8192 tokens
        dict(name="ln_ffn", op="ln_fwd", rows=8192, hidden=7168, dtype="bf16", params="bf16", pad=0, stats=True),
        # an odd width inside a wider buffer, fp16 activations with fp32 parameters
        dict(name="ln_odd_fp16", op="ln_fwd", rows=4097, hidden=1023, dtype="fp16", params="fp32", pad=2, stats=True),
        # its backward pass in training, with the parameters' gradients
        dict(name="ln_bwd_ffn", op="ln_bwd", rows=8192, hidden=7168, dtype="bf16", params="bf16", pad=0),
        # a wide fp32 residual stream, few tokens
        dict(name="ln_bwd_wide_fp32", op="ln_bwd", rows=515, hidden=16384, dtype="fp32", params="fp32", pad=0),
        # one token of a serving step: the weights' bytes are what it has to read
        dict(name="gated_token", op="gated", M=1, K=7168, F=18432, act="silu", bias=False, aux=False),
        # a small model's feed-forward in training, with biases
        dict(name="gated_fc1", op="gated", M=4096, K=1024, F=4096, act="gelu", bias=True, aux=True),
        # the large dense FFN in training
        dict(name="gated_ffn", op="gated", M=8192, K=7168, F=18432, act="silu", bias=False, aux=True),
        # 128 experts, 8 of them for each token, popularity by a power law, some without tokens
        dict(name="gated_moe", op="moe", tokens=16384, top_k=8, experts=128, K=4096, F=768, act="silu", aux=True),
        # the activation's backward pass alone, for recipes that quantise otherwise
        dict(name="gated_bwd_act", op="gated_bwd_act", M=4096, F=4096, act="silu"),
        # gradients of a small batch whose token count fills no tile
        dict(name="gated_bwd_ragged", op="gated_bwd", M=1000, K=1024, F=4096, act="gelu"),
        # gradients of the large dense FFN
        dict(name="gated_bwd_ffn", op="gated_bwd", M=8192, K=7168, F=18432, act="silu"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ln_fwd", "ln_bwd", "gated", "gated", "moe", "gated_bwd_act", "gated_bwd"])
    if op in ("ln_fwd", "ln_bwd"):
        hidden = _log(rng, 64, 16384)
        hidden = hidden if rng.random() < 0.3 else max(64, hidden // 8 * 8)      # odd widths among them
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        rows = _log(rng, 1, min(16384, 8192 * 7168 // hidden // (2 if dtype == "fp32" else 1)))
        c = dict(op=op, rows=rows, hidden=hidden, dtype=dtype, params=rng.choice([dtype, "fp32"]),
                 pad=rng.choice([0, 0, 8, 24]))
        return dict(c, stats=rng.random() < 0.7) if op == "ln_fwd" else c
    act = rng.choice(["silu", "gelu", "relu"])
    K = 128 * _log(rng, 4, 56)
    if op == "gated":
        return dict(op=op, M=_log(rng, 1, 8192), K=K, F=16 * _log(rng, 16, 1152), act=act, bias=rng.random() < 0.4,
                    aux=rng.random() < 0.6)
    if op == "moe":
        return dict(op=op, tokens=_log(rng, 16, 8192), top_k=rng.choice([1, 2, 4, 8]), experts=rng.choice([8, 16, 64, 128]),
                    K=128 * _log(rng, 4, 32), F=16 * _log(rng, 16, 48), act=act, aux=rng.random() < 0.6)
    if op == "gated_bwd_act":
        return dict(op=op, M=_log(rng, 1, 8192), F=16 * _log(rng, 16, 1152), act=act)
    return dict(op=op, M=_log(rng, 1, 8192), K=K, F=64 * _log(rng, 4, 288), act=act)


def work(case):
    c = case
    if c["op"] in ("ln_fwd", "ln_bwd"):
        n, b, p = c["rows"] * c["hidden"], DTYPES[c["dtype"]].itemsize, DTYPES[c["params"]].itemsize
        if c["op"] == "ln_fwd":
            return {"bytes": 2 * n * b + 2 * c["hidden"] * p + (8 * c["rows"] if c["stats"] else 0), "flops": 8 * n}
        return {"bytes": 3 * n * b + 3 * c["hidden"] * p + 8 * c["rows"], "flops": 14 * n}
    F = c["F"]
    if c["op"] == "gated_bwd_act":
        return {"bytes": 10 * c["M"] * F, "flops": 10 * c["M"] * F}
    codes = 33 / 32                                      # a code and its share of a scale
    if c["op"] == "moe":
        M, K, touched = c["tokens"] * c["top_k"], c["K"], min(c["experts"], c["tokens"] * c["top_k"])
        return {"bytes": codes * (M * K + touched * 2 * F * K) + 2 * M * F * (3 if c["aux"] else 1), "flops": 4 * M * F * K}
    M, K = c["M"], c["K"]
    if c["op"] == "gated":
        return {"bytes": codes * (M * K + 2 * F * K) + 2 * M * F * (3 if c["aux"] else 1), "flops": 4 * M * F * K}
    return {"bytes": 6 * M * F + codes * (M * K + 2 * F * K) + 2 * M * K + 4 * F * K, "flops": 8 * M * F * K}


# ------------------------------------------------------------------ inputs

def _up(n, m):
    return (n + m - 1) // m * m


def _encode(x):
    """MXFP8 codes and scale bytes of a matrix, 32 elements of a row to a scale
    (rows of scales padded to 16 bytes): what a program holds of its operands."""
    rows, cols = x.shape
    b = x.float().reshape(rows, cols // 32, 32)
    e = (torch.frexp(b.abs().amax(2))[1] - 9).clamp(-127, 127)          # floor(log2 amax) - 8
    q = torch.ldexp(b, -e[:, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    s = torch.zeros(rows, _up(cols // 32, 16), dtype=torch.uint8, device=x.device)
    s[:, :cols // 32] = (e + 127).to(torch.uint8)
    return q.reshape(rows, cols).view(torch.uint8), s


def _normal(g, shape, std, mean=0.0):
    return (torch.randn(shape, generator=g, device="cuda") * std + mean).to(torch.bfloat16)


def _activations(g, rows, cols):
    """N(0,1) with 1 in 128 columns 32 times as large, as activations have them."""
    x = torch.randn((rows, cols), generator=g, device="cuda")
    x[:, torch.randperm(cols, generator=g, device="cuda")[:max(1, cols // 128)]] *= 32
    return x.to(torch.bfloat16)


def _pitched(x, pad):
    """x inside a buffer whose rows are `pad` elements longer."""
    if not pad:
        return x
    w = torch.zeros(x.shape[0], x.shape[1] + pad, dtype=x.dtype, device=x.device)
    w[:, :x.shape[1]] = x
    return w[:, :x.shape[1]]


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + 17)
    randn = lambda *shape: torch.randn(shape, generator=g, device="cuda")  # noqa: E731
    if c["op"] in ("ln_fwd", "ln_bwd"):
        R, H, t, p = c["rows"], c["hidden"], DTYPES[c["dtype"]], DTYPES[c["params"]]
        x = randn(R, H) * torch.exp2(2 * torch.rand((R, 1), generator=g, device="cuda") - 1) + 0.5 * randn(R, 1)
        s = dict(c, x=_pitched(x.to(t), c["pad"]), gamma=(1 + 0.1 * randn(H)).to(p), beta=(0.1 * randn(H)).to(p))
        if c["op"] == "ln_bwd":
            s["dy"] = _pitched((0.01 * randn(R, H)).to(t), c["pad"])
            v = s["x"].double()                          # saved by the forward pass
            mu = v.mean(1, keepdim=True)
            s["mu"] = mu[:, 0].float()
            s["rsigma"] = ((v - mu).square().mean(1) + EPS).rsqrt().float()
        return s
    F = c["F"]
    if c["op"] == "gated_bwd_act":
        return dict(c, dh=_normal(g, (c["M"], F), 1e-3), gate_up=_normal(g, (c["M"], 2 * F), 1.5))
    K = c["K"]
    if c["op"] == "moe":
        T, k, E = c["tokens"], c["top_k"], c["experts"]
        p = torch.arange(1, E + 1, dtype=torch.float64, device="cuda") ** -1.1
        p = p[torch.randperm(E, generator=g, device="cuda")]
        if E > 4 * k:
            p[torch.randperm(E, generator=g, device="cuda")[:E // 32]] = 0
        noise = -torch.log(-torch.log(torch.rand((T, E), generator=g, device="cuda", dtype=torch.float64)))
        picks = torch.topk(p.log()[None, :] + noise, k, dim=1).indices
        m = torch.bincount(picks.flatten(), minlength=E)
        qx, sx = _encode(_activations(g, T * k, K))
        qw, sw = _encode(_normal(g, (E * 2 * F, K), 0.02))
        return dict(c, qx=qx, sx=sx, qw=qw.view(E, 2 * F, K), sw=sw, group_m=m.to(torch.int32), sizes=m.tolist())
    M = c["M"]
    if c["op"] == "gated":
        qx, sx = _encode(_activations(g, M, K))
        qw, sw = _encode(_normal(g, (2 * F, K), 0.02))
        return dict(c, qx=qx, sx=sx, qw=qw, sw=sw, b=_normal(g, (2 * F,), 0.02) if c["bias"] else None)
    # the column-wise copies of W and of X that a training program has from the forward pass
    x = torch.zeros(_up(M, 128), K, dtype=torch.bfloat16, device="cuda")
    x[:M] = _activations(g, M, K)
    qx, sx = _encode(x.t().contiguous())
    qw, sw = _encode(_normal(g, (K, 2 * F), 0.02))
    return dict(c, dh=_normal(g, (M, F), 1e-3), gate_up=_normal(g, (M, 2 * F), 1.5), qx=qx, sx=sx, qw=qw, sw=sw)


# ------------------------------------------------------------------ the plain form

def _decode(q, s):
    rows, cols = q.shape
    v = q.view(torch.float8_e4m3fn).float().reshape(rows, cols // 32, 32)
    return torch.ldexp(v, s[:, :cols // 32, None].int() - 127).reshape(rows, cols)


def _act(x, act):
    if act == "relu":
        return torch.where(x > 0, x, torch.zeros_like(x))
    if act == "silu":
        return x / (1 + torch.exp(-x))
    return 0.5 * x * (1 + torch.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x * x * x)))


def _act_grad(x, act):
    if act == "relu":
        return (x > 0).to(x.dtype)
    if act == "silu":
        s = 1 / (1 + torch.exp(-x))
        return s * (1 + x * (1 - s))
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (x + 0.044715 * x * x * x))
    return 0.5 * (1 + t) + 0.5 * x * (1 - t * t) * c * (1 + 3 * 0.044715 * x * x)


def _plain_gated(x, w, b, act):
    gu = x @ w.t()
    if b is not None:
        gu = gu + b.float()
    F = gu.shape[1] // 2
    return (_act(gu[:, :F], act) * gu[:, F:]).to(torch.bfloat16), gu.to(torch.bfloat16)


def _plain_dgated(s):
    F, dh, gu = s["F"], s["dh"].float(), s["gate_up"].float()
    g, u = gu[:, :F], gu[:, F:]
    return torch.cat([dh * u * _act_grad(g, s["act"]), dh * _act(g, s["act"])], 1).to(torch.bfloat16)


def _plain(s):
    op = s["op"]
    if op == "ln_fwd":
        x = s["x"].float()
        mu = x.mean(1, keepdim=True)
        d = x - mu
        rs = 1 / torch.sqrt((d * d).mean(1, keepdim=True) + EPS)
        y = (d * rs * s["gamma"].float() + s["beta"].float()).to(s["x"].dtype)
        return {"y": y, "mu": mu[:, 0], "rsigma": rs[:, 0]} if s["stats"] else {"y": y}
    if op == "ln_bwd":
        dy, rs = s["dy"].float(), s["rsigma"][:, None]
        xh = (s["x"].float() - s["mu"][:, None]) * rs
        g = dy * s["gamma"].float()
        dx = rs * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
        p = s["gamma"].dtype
        return {"dx": dx.to(s["x"].dtype), "dgamma": (dy * xh).sum(0).to(p), "dbeta": dy.sum(0).to(p)}
    if op == "gated":
        h, gu = _plain_gated(_decode(s["qx"], s["sx"]), _decode(s["qw"], s["sw"]), s["b"], s["act"])
        return {"h": h, "gate_up": gu} if s["aux"] else {"h": h}
    if op == "moe":
        E, N, K = s["qw"].shape
        x, w = _decode(s["qx"], s["sx"]).split(s["sizes"]), _decode(s["qw"].view(E * N, K), s["sw"]).view(E, N, K)
        parts = [_plain_gated(x[e], w[e], None, s["act"]) for e in range(E)]          # experts differ in their rows
        h, gu = (torch.cat([p[i] for p in parts]) for i in (0, 1))
        return {"h": h, "gate_up": gu} if s["aux"] else {"h": h}
    d = _plain_dgated(s)
    if op == "gated_bwd_act":
        return {"d_gate_up": d}
    dt = torch.zeros(d.shape[1], s["qx"].shape[1], dtype=d.dtype, device=d.device)
    dt[:, :s["M"]] = d.t()
    dx = _decode(*_encode(d)) @ _decode(s["qw"], s["sw"]).t()
    dw = _decode(*_encode(dt)) @ _decode(s["qx"], s["sx"]).t()
    return {"dx": dx.to(torch.bfloat16), "dw": dw.to(torch.bfloat16)}


# ------------------------------------------------------------------ the framework's calls

def run(state):
    s = state
    if not own:
        return _plain(s)
    import mxfp8_block_scaled_quantize_gb300 as temx
    op = s["op"]
    if op == "ln_fwd":
        return temx.layernorm(s["x"], s["gamma"], s["beta"], eps=EPS, stats=s["stats"])
    if op == "ln_bwd":
        return temx.layernorm_backward(s["dy"], s["x"], s["gamma"], s["mu"], s["rsigma"])
    if op == "gated":
        h, gu = temx.gated_gemm(s["qx"], s["sx"], s["qw"], s["sw"], activation=s["act"], bias=s["b"], aux=s["aux"])
        return {"h": h, "gate_up": gu} if s["aux"] else {"h": h}
    if op == "moe":
        h, gu = temx.grouped_gated_gemm(s["group_m"], s["qx"], s["sx"], s["qw"], s["sw"], activation=s["act"],
                                        aux=s["aux"])
        return {"h": h, "gate_up": gu} if s["aux"] else {"h": h}
    if op == "gated_bwd_act":
        return temx.gated_backward(s["dh"], s["gate_up"], activation=s["act"], dense=True, rowwise=False, colwise=False)
    d = temx.gated_backward(s["dh"], s["gate_up"], activation=s["act"], rowwise=True, colwise=True)
    dx, _ = temx.gemm(d["q_row"], d["s_row"], s["qw"], s["sw"])
    dw, _ = temx.gemm(d["q_col"], d["s_col"], s["qx"], s["sx"])
    return {"dx": dx, "dw": dw}


# ------------------------------------------------------------------ the definition in 64 bits

def _value64(q, s):
    """Codes and scales as numbers, from the formats' fields."""
    c = q.long()
    field, frac = (c >> 3) & 15, (c & 7).double()
    mag = torch.where(field == 0, frac / 8 * 2.0 ** -6, (1 + frac / 8) * torch.exp2((field - 7).double()))
    v = torch.where(c >= 128, -mag, mag)
    return v * torch.exp2(s[:, :q.shape[1] // 32].double() - 127).repeat_interleave(32, 1)


def _nearest(v, bits, lowest):
    """v rounded to `bits` fraction bits, ties to even, exponents from `lowest` on."""
    _, e = torch.frexp(v)
    unit = torch.exp2((torch.clamp(e - 1, min=lowest) - bits).double())
    return torch.round(v / unit) * unit


def _mx64(v):
    """The values that MXFP8 keeps of a matrix, 32 of a row to a scale."""
    b = v.reshape(v.shape[0], -1, 32)
    _, e = torch.frexp(b.abs().amax(2, keepdim=True))
    unit = torch.exp2(torch.clamp(e - 9, -127, 127).double())
    return (torch.clamp(_nearest(b / unit, 3, -6), -448, 448) * unit).reshape(v.shape)


def _sigmoid64(x):
    return torch.where(x >= 0, 1 / (1 + torch.exp(-x.abs())), torch.exp(-x.abs()) / (1 + torch.exp(-x.abs())))


def _act64(x, act):
    """(act(x), act'(x))"""
    if act == "relu":
        return x.clamp(min=0), (x > 0).double()
    if act == "silu":
        p = _sigmoid64(x)
        return x * p, p + x * p * _sigmoid64(-x)
    a = 2 * math.sqrt(2 / math.pi)                        # (1 + tanh z) / 2 is the logistic function of 2z
    z = a * (x + 0.044715 * x ** 3)
    p = _sigmoid64(z)
    return x * p, p + x * p * _sigmoid64(-z) * a * (1 + 0.134145 * x * x)


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "ln_fwd":
        x = s["x"].double()
        n = x.shape[1]
        mu = x.sum(1) / n
        d = x - mu[:, None]
        rs = (d.pow(2).sum(1) / n + EPS).pow(-0.5)
        y = s["gamma"].double() * (d * rs[:, None]) + s["beta"].double()
        return {"y": y, "mu": mu, "rsigma": rs} if s["stats"] else {"y": y}
    if op == "ln_bwd":
        x, dy, rs = s["x"].double(), s["dy"].double(), s["rsigma"].double()
        n = x.shape[1]
        xh = (x - s["mu"].double()[:, None]).mul_(rs[:, None])
        w = dy * s["gamma"].double()
        c = torch.stack([w.sum(1), torch.einsum("rh,rh->r", w, xh)]) / n
        return {"dx": (w - c[0, :, None] - xh * c[1, :, None]) * rs[:, None],
                "dgamma": torch.einsum("rh,rh->h", dy, xh), "dbeta": dy.sum(0)}
    if op in ("gated", "moe"):
        F = s["F"]
        if op == "gated":
            gu = _value64(s["qx"], s["sx"]) @ _value64(s["qw"], s["sw"]).T
            gu = gu if s["b"] is None else gu + s["b"].double()
        else:
            N, K = s["qw"].shape[1:]
            gu, r = torch.empty(s["qx"].shape[0], N, dtype=torch.float64, device="cuda"), 0
            for e, m in enumerate(s["sizes"]):
                w = _value64(s["qw"][e], s["sw"][e * N:(e + 1) * N])
                gu[r:r + m] = _value64(s["qx"][r:r + m], s["sx"][r:r + m]) @ w.T
                r += m
        h = _act64(gu[:, :F], s["act"])[0] * gu[:, F:]
        return {"h": h, "gate_up": gu} if s["aux"] else {"h": h}
    F, dh, gu = s["F"], s["dh"].double(), s["gate_up"].double()
    a, da = _act64(gu[:, :F], s["act"])
    d = torch.empty(dh.shape[0], 2 * F, dtype=torch.float64, device="cuda")
    d[:, :F], d[:, F:] = dh * gu[:, F:] * da, dh * a
    if op == "gated_bwd_act":
        return {"d_gate_up": d}
    d = _nearest(d, 7, -126)                              # bf16, by the operator's definition
    dx = _mx64(d) @ _value64(s["qw"], s["sw"]).T
    tokens = s["qx"].shape[1]
    dt = torch.zeros(2 * F, tokens, dtype=torch.float64, device="cuda")
    dt[:, :dh.shape[0]] = d.T
    return {"dx": dx, "dw": _mx64(dt) @ _value64(s["qx"], s["sx"]).T}

"""Cases for the operators around a mixture-of-experts feed-forward: inputs, a
plain form in elementary torch operations, and the framework's calls.

Operators (a row is a token; T tokens, k experts for each, E experts):

* RMSNorm with the residual's addition: z = x + residual, rounded to its type,
  rsigma = 1/sqrt(mean(z^2) + eps), y = z rsigma gamma; y in the activations'
  type, or MXFP8 (E4M3 codes, one E8M0 scale per 32) row-wise and column-wise.
  Backward: xh = z rsigma, g = dy gamma, dx = rsigma (g - xh mean(g xh)) + dz,
  dgamma = sum over the rows of dy xh.
* Router: the k experts with the largest logit + bias of a row, in falling order
  (ties to the lowest index), and their weights, scale * softmax or sigmoid of
  the logits, renormalised over the chosen ones or not; and the logits' gradient
  from the weights'.
* Tokens sorted by expert: slot t k + j of index [T, k] goes to the row that a
  stable sort by expert gives it (slots with index -1, a batch's padding, have
  none); the experts' row counts; every token's row copied to its slots' rows, in
  its type or as MXFP8 codes and scales.
* And back: out[t] = residual[t] + sum_j weight[t, j] y[row[t, j]].  Backward:
  dy[row[t, j]] = weight[t, j] dout[t], dweight[t, j] = <dout[t], y[row[t, j]]>.
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
        dict(name="rms_token", op="rms", rows=1, hidden=7168, dtype="bf16", params="bf16", residual=True, pad=0),
        # an odd width inside a wider buffer, fp16 activations with fp32 parameters
        dict(name="rms_odd_fp16", op="rms", rows=3001, hidden=1021, dtype="fp16", params="fp32", residual=True, pad=3),
        # the large dense FFN's norm in the backward pass, the residual path's gradient added
        dict(name="rms_bwd_ffn", op="rms_bwd", rows=8192, hidden=7168, dtype="bf16", params="bf16", dz=True, pad=0),
        # a wide fp32 residual stream, few tokens
        dict(name="rms_bwd_fp32", op="rms_bwd", rows=1111, hidden=8200, dtype="fp32", params="fp32", dz=False, pad=0),
        # a training step of the large dense FFN: the input of its GEMMs, both ways
        dict(name="rmsq_ffn", op="rmsq", rows=8192, hidden=7168, params="bf16", residual=True, colwise=True, dense=False),
        # a batch of single tokens in serving: the experts' operand, and the router's
        dict(name="rmsq_decode", op="rmsq", rows=48, hidden=4096, params="bf16", residual=True, colwise=False, dense=True),
        # routing of a training step, 8 of 128 experts, with the logits' gradient
        dict(name="route_train", op="route", tokens=16384, experts=128, k=8, dtype="bf16", scoring="softmax",
             renormalise=True, scale=1.0, bias=False, backward=True),
        # routing of a batch of single tokens, the choice balanced by a bias
        dict(name="route_decode", op="route", tokens=33, experts=64, k=6, dtype="fp32", scoring="sigmoid",
             renormalise=True, scale=2.5, bias=True, backward=False),
        # the experts' rows of a training step
        dict(name="dispatch_moe", op="dispatch", tokens=16384, k=8, experts=128, hidden=4096, dtype="bf16", padding=0),
        # a small serving batch with padding, quantised once for all its experts
        dict(name="dispatch_mx_small", op="dispatch", tokens=100, k=4, experts=64, hidden=2048, dtype="mx", padding=3),
        # the experts' outputs of a training step, added to the residual
        dict(name="combine_moe", op="combine", tokens=16384, k=8, experts=128, hidden=4096, dtype="bf16", padding=0,
             weights=True, residual=True),
        # its gradients in a smaller model
        dict(name="combine_bwd_fp16", op="combine_bwd", tokens=4099, k=6, experts=64, hidden=2048, dtype="fp16", padding=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rms", "rms_bwd", "rmsq", "route", "dispatch", "combine", "combine_bwd"])
    if op in ("rms", "rms_bwd"):
        hidden = _log(rng, 64, 16384)
        hidden = hidden if rng.random() < 0.3 else max(64, hidden // 8 * 8)      # odd widths among them
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        rows = _log(rng, 1, min(16384, 8192 * 7168 // hidden // (2 if dtype == "fp32" else 1)))
        c = dict(op=op, rows=rows, hidden=hidden, dtype=dtype, params=rng.choice([dtype, "fp32"]),
                 pad=rng.choice([0, 0, 8, 24]))
        return dict(c, **{"residual" if op == "rms" else "dz": rng.random() < 0.7})
    if op == "rmsq":
        colwise = rng.random() < 0.5
        rows = 32 * _log(rng, 1, 256) if colwise else _log(rng, 1, 8192)
        return dict(op=op, rows=rows, hidden=32 * _log(rng, 4, 224), params=rng.choice(["bf16", "fp32"]),
                    residual=rng.random() < 0.7, colwise=colwise, dense=rng.random() < 0.3)
    k = rng.choice([1, 2, 4, 6, 8])
    experts = rng.choice([8, 16, 60, 64, 128, 160, 256])
    if op == "route":
        return dict(op=op, tokens=_log(rng, 1, 16384), experts=experts, k=k, dtype=rng.choice(["bf16", "fp32", "fp16"]),
                    scoring=rng.choice(["softmax", "sigmoid"]), renormalise=rng.random() < 0.6,
                    scale=rng.choice([1.0, 2.5]), bias=rng.random() < 0.4, backward=rng.random() < 0.6)
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"] + (["mx", "mx"] if op == "dispatch" else []))
    hidden = 128 * _log(rng, 2, 56) if dtype == "mx" else 8 * _log(rng, 32, 896)
    hidden += 0 if dtype == "mx" or rng.random() < 0.8 else rng.randrange(1, 8)  # rows off 16-byte boundaries
    tokens = _log(rng, 1, max(2, min(16384, 16384 * 8 * 4096 // (k * hidden * (2 if dtype == "fp32" else 1)))))
    c = dict(op=op, tokens=tokens, k=k, experts=experts, hidden=hidden, dtype=dtype,
             padding=rng.choice([0, 0, tokens // 10]))
    return dict(c, weights=rng.random() < 0.7, residual=rng.random() < 0.5) if op == "combine" else c


def work(case):
    c = case
    op = c["op"]
    if op in ("rms", "rms_bwd", "rmsq"):
        n = c["rows"] * c["hidden"]
        b, p = DTYPES[c.get("dtype", "bf16")].itemsize, DTYPES[c["params"]].itemsize
        side = c["hidden"] * p + 4 * c["rows"]
        if op == "rms":
            return {"bytes": n * b * (4 if c["residual"] else 2) + side, "flops": 5 * n}
        if op == "rms_bwd":
            return {"bytes": n * b * (4 if c["dz"] else 3) + side + c["hidden"] * p, "flops": 10 * n}
        copies = n * 33 / 32 * (2 if c["colwise"] else 1) + (n * b if c["dense"] else 0)
        return {"bytes": n * b * (3 if c["residual"] else 1) + copies + side, "flops": 8 * n}
    T, k = c["tokens"], c["k"]
    if op == "route":
        b = DTYPES[c["dtype"]].itemsize * T * c["experts"]
        return {"bytes": b * (2 if c["backward"] else 1) + T * k * (12 if c["backward"] else 8), "flops": 6 * T * c["experts"]}
    H, rows = c["hidden"], (T - c["padding"]) * k
    b = 33 / 32 if c["dtype"] == "mx" else DTYPES[c["dtype"]].itemsize
    if op == "dispatch":
        return {"bytes": H * b * (T - c["padding"] + rows) + 12 * T * k + 4 * c["experts"], "flops": T * k}
    if op == "combine":
        return {"bytes": H * b * (rows + T * (2 if c["residual"] else 1)) + T * k * (8 if c["weights"] else 4),
                "flops": 2 * rows * H}
    return {"bytes": H * b * (2 * rows + T - c["padding"]) + 12 * T * k, "flops": 3 * rows * H}


# ------------------------------------------------------------------ inputs

def _pitched(x, pad):
    """x inside a buffer whose rows are `pad` elements longer."""
    if not pad:
        return x
    w = torch.zeros(x.shape[0], x.shape[1] + pad, dtype=x.dtype, device=x.device)
    w[:, :x.shape[1]] = x
    return w[:, :x.shape[1]]


def _encode(x):
    """MXFP8 codes and scale bytes of a matrix, 32 elements of a row to a scale
    (rows of scales padded to 16 bytes)."""
    rows, cols = x.shape
    b = x.float().reshape(rows, cols // 32, 32)
    e = (torch.frexp(b.abs().amax(2))[1] - 9).clamp(-127, 127)          # floor(log2 amax) - 8
    q = torch.ldexp(b, -e[:, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    s = torch.zeros(rows, (cols // 32 + 15) // 16 * 16, dtype=torch.uint8, device=x.device)
    s[:, :cols // 32] = (e + 127).to(torch.uint8)
    return q.reshape(rows, cols).view(torch.uint8), s


def _choices(g, T, k, E, padding):
    """Experts by a power law, distinct for a token; -1 for the padding at the batch's end."""
    p = torch.arange(1, E + 1, dtype=torch.float64, device="cuda") ** -1.1
    p = p[torch.randperm(E, generator=g, device="cuda")]
    noise = -torch.log(-torch.log(torch.rand((T, E), generator=g, device="cuda", dtype=torch.float64)))
    index = torch.topk(p.log()[None, :] + noise, k, dim=1).indices.to(torch.int32)
    index[T - padding:] = -1
    return index


def _rows_of(index, E):
    """The row of each slot (-1: none), from the experts' sorted slots."""
    flat = index.flatten().long()
    order = torch.sort(torch.where(flat < 0, E, flat), stable=True).indices
    row = torch.empty_like(flat)
    row[order] = torch.arange(flat.numel(), device=flat.device)
    return torch.where(flat < 0, -1, row).to(torch.int32).view(index.shape)


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed * 6007 + 23)
    randn = lambda *shape: torch.randn(shape, generator=g, device="cuda")  # noqa: E731
    op = c["op"]
    if op in ("rms", "rms_bwd", "rmsq"):
        R, H, t, p = c["rows"], c["hidden"], DTYPES[c.get("dtype", "bf16")], DTYPES[c["params"]]
        wide = torch.ones(H, device="cuda")                             # a few channels are much larger
        wide[torch.randperm(H, generator=g, device="cuda")[:max(1, H // 128)]] = 16
        stream = randn(R, H) * wide * torch.exp2(2 * torch.rand((R, 1), generator=g, device="cuda") - 1)
        s = dict(c, gamma=(1 + 0.1 * randn(H)).to(p))
        pad = c.get("pad", 0)
        if op == "rms_bwd":
            s["z"], s["dy"] = _pitched(stream.to(t), pad), _pitched((0.01 * randn(R, H)).to(t), pad)
            s["dz"] = _pitched((0.02 * randn(R, H)).to(t), pad) if c["dz"] else None
            s["rsigma"] = (s["z"].double().square().mean(1) + EPS).rsqrt().float()      # saved by the forward pass
            return s
        s["x"] = _pitched((0.5 * randn(R, H) if c["residual"] else stream).to(t), pad)
        s["residual"] = _pitched(stream.to(t), pad) if c["residual"] else None
        return s
    T, k, E = c["tokens"], c["k"], c["experts"]
    if op == "route":
        logits = (randn(T, E) + 0.5 * randn(1, E)).to(DTYPES[c["dtype"]])
        return dict(c, logits=logits, bias=0.2 * randn(E) if c["bias"] else None, dweight=randn(T, k))
    index = _choices(g, T, k, E, c["padding"])
    H, kept = c["hidden"], (T - c["padding"]) * k
    if op == "dispatch":
        if c["dtype"] == "mx":
            x, scales = _encode(randn(T, H))
            return dict(c, index=index, x=x, scales=scales, kept=kept)
        return dict(c, index=index, x=randn(T, H).to(DTYPES[c["dtype"]]), scales=None, kept=kept)
    t = DTYPES[c["dtype"]]
    s = dict(c, row=_rows_of(index, E), y=randn(T * k, H).to(t))
    w = torch.rand((T, k), generator=g, device="cuda") + 0.05
    s["weight"] = w / w.sum(1, keepdim=True) if op == "combine_bwd" or c["weights"] else None
    if op == "combine":
        s["residual"] = randn(T, H).to(t) if c["residual"] else None
    else:
        s["dout"] = (0.01 * randn(T, H)).to(t)
    s["kept"] = kept
    return s


# ------------------------------------------------------------------ the plain form

def _plain_norm(s):
    x = s["x"]
    z = x if s["residual"] is None else (x.float() + s["residual"].float()).to(x.dtype)
    f = z.float()
    rs = 1 / torch.sqrt((f * f).mean(1, keepdim=True) + EPS)
    return z, rs[:, 0], f * rs * s["gamma"].float()


def _mx_out(out, name, q, s, blocks):
    """Codes and scales as the numbers that they stand for."""
    out["q_" + name] = q.view(torch.float8_e4m3fn)
    out["s_" + name] = s[:, :blocks].view(torch.float8_e8m0fnu)


def _score(l, s):
    """exp(l - max) and its sum, or the logistic function, of a row's logits."""
    if s["scoring"] == "softmax":
        e = torch.exp(l - l.amax(1, keepdim=True))
        return e / e.sum(1, keepdim=True)
    return 1 / (1 + torch.exp(-l))


def _plain_route(s):
    l = s["logits"].float()
    key = l if s["bias"] is None else l + s["bias"]
    index = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :s["k"]]
    p = _score(l, s)
    c = p.gather(1, index)
    total = c.sum(1, keepdim=True) if s["renormalise"] else torch.ones_like(c[:, :1])
    w = c / total
    out = {"index": index.to(torch.int32), "weight": w * s["scale"]}
    if s["backward"]:
        g = s["dweight"] * s["scale"]
        if s["renormalise"]:                                            # of the chosen scores
            g = (g - (g * w).sum(1, keepdim=True)) / total
        dp = torch.zeros_like(p).scatter(1, index, g)
        if s["scoring"] == "softmax":
            d = p * (dp - (dp * p).sum(1, keepdim=True))
        else:
            d = dp * p * (1 / (1 + torch.exp(l)))
        out["dlogits"] = d.to(s["logits"].dtype)
    return out


def _plain_dispatch(s):
    flat, E, n = s["index"].flatten().long(), s["experts"], s["index"].numel()
    by, order = torch.sort(torch.where(flat < 0, E, flat), stable=True)
    at = torch.arange(n, device=flat.device)
    row = torch.empty_like(flat)
    row[order] = at
    ends = torch.searchsorted(by, torch.arange(E + 1, device=flat.device))
    out = {"group_m": (ends[1:] - ends[:-1]).to(torch.int32),
           "row": torch.where(flat < 0, -1, row).to(torch.int32).view(s["index"].shape),
           "slot": torch.where(by < E, order, -1).to(torch.int32)}
    token = torch.div(order[:s["kept"]], s["k"], rounding_mode="floor")
    if s["scales"] is None:
        return dict(out, x=s["x"][token])
    _mx_out(out, "row", s["x"][token], s["scales"][token], s["hidden"] // 32)
    return out


def _plain(s):
    op = s["op"]
    if op == "rms":
        z, rs, y = _plain_norm(s)
        out = {"y": y.to(z.dtype), "rsigma": rs}
        return out if s["residual"] is None else dict(out, z=z)
    if op == "rmsq":
        z, rs, y = _plain_norm(s)
        out = {"rsigma": rs} if s["residual"] is None else {"rsigma": rs, "z": z}
        _mx_out(out, "row", *_encode(y), s["hidden"] // 32)
        if s["colwise"]:
            _mx_out(out, "col", *_encode(y.t()), s["rows"] // 32)
        return dict(out, y=y.to(z.dtype)) if s["dense"] else out
    if op == "rms_bwd":
        dy, rs = s["dy"].float(), s["rsigma"][:, None]
        xh = s["z"].float() * rs
        g = dy * s["gamma"].float()
        dx = rs * (g - xh * (g * xh).mean(1, keepdim=True))
        dx = dx if s["dz"] is None else dx + s["dz"].float()
        return {"dx": dx.to(s["z"].dtype), "dgamma": (dy * xh).sum(0).to(s["gamma"].dtype)}
    if op == "route":
        return _plain_route(s)
    if op == "dispatch":
        return _plain_dispatch(s)
    T, k = s["row"].shape
    live = (s["row"] >= 0)[:, :, None]
    rows = s["row"].clamp(min=0).long()
    picked = torch.where(live, s["y"][rows].float(), 0.0)
    if op == "combine":
        if s["weight"] is not None:
            picked = picked * s["weight"][:, :, None]
        out = picked.sum(1)
        return {"out": (out if s["residual"] is None else out + s["residual"].float()).to(s["y"].dtype)}
    dout = s["dout"].float()[:, None, :]
    dy = torch.empty_like(s["y"])
    dy[rows[:T - s["padding"]]] = (dout * s["weight"][:, :, None]).to(dy.dtype)[:T - s["padding"]]
    return {"dy": dy[:s["kept"]], "dweight": (picked * dout).sum(2)}


# ------------------------------------------------------------------ the framework's calls

def run(state):
    s = state
    if not own:
        return _plain(s)
    import mxfp8_block_scaled_quantize_gb300 as temx
    op = s["op"]
    if op == "rms":
        return temx.rmsnorm(s["x"], s["gamma"], eps=EPS, residual=s["residual"])
    if op == "rmsq":
        r = temx.rmsnorm_quantize(s["x"], s["gamma"], eps=EPS, residual=s["residual"], colwise=s["colwise"],
                                  dense=s["dense"])
        out = {n: r[n] for n in ("rsigma", "z", "y") if n in r}
        _mx_out(out, "row", r["q_row"], r["s_row"], s["hidden"] // 32)
        if s["colwise"]:
            _mx_out(out, "col", r["q_col"], r["s_col"], s["rows"] // 32)
        return out
    if op == "rms_bwd":
        return temx.rmsnorm_backward(s["dy"], s["z"], s["gamma"], s["rsigma"], dz=s["dz"])
    if op == "route":
        how = dict(scoring=s["scoring"], renormalise=s["renormalise"], scale=s["scale"])
        out = temx.route(s["logits"], s["k"], bias=s["bias"], **how)
        if s["backward"]:
            out["dlogits"] = temx.route_backward(s["dweight"], s["logits"], out["index"], **how)
        return out
    if op == "dispatch":
        out = temx.moe_sort(s["index"], s["experts"])
        if s["scales"] is None:
            out["x"] = temx.moe_dispatch(s["x"], out["row"])[:s["kept"]]
            return out
        q, scales = temx.moe_dispatch(s["x"], out["row"], scales=s["scales"])
        _mx_out(out, "row", q[:s["kept"]], scales[:s["kept"]], s["hidden"] // 32)
        return out
    if op == "combine":
        return {"out": temx.moe_combine(s["y"], s["row"], weight=s["weight"], residual=s["residual"])}
    out = temx.moe_combine_backward(s["dout"], s["y"], s["row"], s["weight"])
    return {"dy": out["dy"][:s["kept"]], "dweight": out["dweight"]}


# ------------------------------------------------------------------ the definition in 64 bits

def _round_to(v, dtype):
    """v (64 bits) rounded to a type's fraction bits, ties to even."""
    bits, lowest = {torch.bfloat16: (7, -126), torch.float16: (10, -14), torch.float32: (23, -126)}[dtype]
    _, e = torch.frexp(v)
    unit = torch.exp2((torch.clamp(e - 1, min=lowest) - bits).double())
    return torch.round(v / unit) * unit


def _mx64(out, name, v):
    """Scales of 32 values of a row each, and the values over them, not yet rounded."""
    b = v.reshape(v.shape[0], -1, 32)
    _, e = torch.frexp(b.abs().amax(2))
    unit = torch.exp2(torch.clamp(e - 9, -127, 127).double())
    out["q_" + name] = torch.clamp(b / unit[:, :, None], -448, 448).reshape(v.shape)
    out["s_" + name] = unit


def _exact_norm(s):
    z = s["x"].double()
    if s["residual"] is not None:
        z = _round_to(z + s["residual"].double(), s["x"].dtype)         # what the next layer reads
    ms = torch.einsum("rh,rh->r", z, z) / z.shape[1]
    rs = (ms + EPS).pow(-0.5)
    return z, rs, torch.einsum("rh,r,h->rh", z, rs, s["gamma"].double())


def _exact_route(s):
    l, T, E, k = s["logits"].double(), s["tokens"], s["experts"], s["k"]
    key = s["logits"].float() if s["bias"] is None else s["logits"].float() + s["bias"]  # one addition, by definition
    key, place = key.clone(), torch.arange(E, device=l.device)
    index = torch.empty(T, k, dtype=torch.int64, device=l.device)
    for j in range(k):
        best = torch.where(key == key.amax(1, keepdim=True), place, E).amin(1)
        index[:, j] = best
        key.scatter_(1, best[:, None], -math.inf)
    if s["scoring"] == "softmax":
        p = torch.exp(l - torch.logsumexp(l, 1, keepdim=True))
        dscore = None
    else:
        p, dscore = torch.sigmoid(l), torch.sigmoid(l) * torch.sigmoid(-l)
    c = torch.stack([p[torch.arange(T, device=l.device), index[:, j]] for j in range(k)], 1)
    S = c.sum(1, keepdim=True)
    out = {"index": index.to(torch.int32), "weight": s["scale"] * (c / S if s["renormalise"] else c)}
    if not s["backward"]:
        return out
    g = s["scale"] * s["dweight"].double()
    dc = g / S - (g * c).sum(1, keepdim=True) / S ** 2 if s["renormalise"] else g        # of c / sum(c)
    d = torch.zeros(T, E, dtype=torch.float64, device=l.device)
    if dscore is not None:
        return dict(out, dlogits=d.scatter_(1, index, dc * dscore.gather(1, index)))
    d.scatter_(1, index, dc * c)
    return dict(out, dlogits=d - p * (dc * c).sum(1, keepdim=True))


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "rms":
        z, rs, y = _exact_norm(s)
        out = {"y": y, "rsigma": rs}
        return out if s["residual"] is None else dict(out, z=s["x"].double() + s["residual"].double())
    if op == "rmsq":
        z, rs, y = _exact_norm(s)
        out = {"rsigma": rs}
        if s["residual"] is not None:
            out["z"] = s["x"].double() + s["residual"].double()
        _mx64(out, "row", y)
        if s["colwise"]:
            _mx64(out, "col", y.T)
        return dict(out, y=y) if s["dense"] else out
    if op == "rms_bwd":
        z, dy, rs = s["z"].double(), s["dy"].double(), s["rsigma"].double()
        xh = z * rs[:, None]
        w = dy * s["gamma"].double()
        dx = rs[:, None] * w - xh * (rs * torch.einsum("rh,rh->r", w, xh) / z.shape[1])[:, None]
        return {"dx": dx if s["dz"] is None else dx + s["dz"].double(), "dgamma": torch.einsum("rh,rh->h", dy, xh)}
    if op == "route":
        return _exact_route(s)
    if op == "dispatch":
        flat = s["index"].flatten().tolist()
        rows = [[] for _ in range(s["experts"])]
        for slot, e in enumerate(flat):
            if e >= 0:
                rows[e].append(slot)
        slots = [i for r in rows for i in r]
        row = [-1] * len(flat)
        for r, i in enumerate(slots):
            row[i] = r
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        out = {"group_m": i32([len(r) for r in rows]), "row": i32(row).view(s["index"].shape),
               "slot": i32(slots + [-1] * (len(flat) - len(slots)))}
        token = torch.tensor([i // s["k"] for i in slots], dtype=torch.int64, device="cuda")
        if s["scales"] is None:
            return dict(out, x=s["x"].double()[token])
        code = s["x"].long()
        field, frac = (code >> 3) & 15, (code & 7).double()
        v = torch.where(field == 0, frac / 8 * 2.0 ** -6, (1 + frac / 8) * torch.exp2((field - 7).double()))
        v = torch.where(code >= 128, -v, v)
        return dict(out, q_row=v[token], s_row=torch.exp2(s["scales"][:, :s["hidden"] // 32].double() - 127)[token])
    T, k = s["row"].shape
    H, y = s["hidden"], s["y"]
    if op == "combine":
        out = torch.zeros(T, H, dtype=torch.float64, device=y.device)
        for j in range(k):
            r = s["row"][:, j].long()
            t = (r >= 0).nonzero()[:, 0]
            v = y[r[t]].double()
            out[t] += v if s["weight"] is None else v * s["weight"][t, j, None].double()
        return {"out": out if s["residual"] is None else out + s["residual"].double()}
    dy = torch.zeros(T * k, H, dtype=torch.float64, device=y.device)
    dw = torch.zeros(T, k, dtype=torch.float64, device=y.device)
    for j in range(k):
        r = s["row"][:, j].long()
        t = (r >= 0).nonzero()[:, 0]
        d = s["dout"][t].double()
        dy[r[t]] = d * s["weight"][t, j, None].double()
        dw[t, j] = torch.einsum("th,th->t", d, y[r[t]].double())
    return {"dy": dy[:s["kept"]], "dweight": dw}

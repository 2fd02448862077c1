"""A pre-norm gated feed-forward block in MXFP8, trained and served.

    y   = W_down (act(W_gate n) * (W_up n)),   n = LayerNorm(x)
    out = LayerNorm(x + y)

Training (tokens a multiple of 128, the granularity of a GEMM's K): the first
LayerNorm goes straight to MXFP8, the gated GEMM keeps its pre-activations, and
the backward pass gives every gradient.  Serving: any number of tokens, one
included, nothing kept.

    python examples/gated_mlp.py [--tokens 4096 --hidden 1024 --ffn 4096]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mxfp8_block_scaled_quantize_gb300 as temx  # noqa: E402


class GatedMLP:
    def __init__(self, hidden: int, ffn: int, activation: str = "silu", seed: int = 0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        bf = torch.bfloat16
        self.activation = activation
        self.norm_in = ((1 + 0.1 * randn(hidden)).to(bf), (0.1 * randn(hidden)).to(bf))
        self.norm_out = ((1 + 0.1 * randn(hidden)).to(bf), (0.1 * randn(hidden)).to(bf))
        self.w_gate_up = (randn(2 * ffn, hidden) * hidden ** -0.5).to(bf)        # gate rows, then up rows
        self.w_down = (randn(hidden, ffn) * ffn ** -0.5).to(bf)
        # both copies of the weights, made once per optimiser step
        self.q_gate_up = temx.quantize(self.w_gate_up, rowwise=True, colwise=True)
        self.q_down = temx.quantize(self.w_down, rowwise=True, colwise=True)

    def forward(self, x):
        """x bf16 [tokens, hidden] -> (out, what the backward pass needs)."""
        n = temx.layernorm_quantize(x, *self.norm_in, rowwise=True, colwise=True)
        h, pre = temx.gated_gemm(n["q_row"], n["s_row"], self.q_gate_up["q_row"], self.q_gate_up["s_row"],
                                 activation=self.activation, aux=True)
        qh = temx.quantize(h, rowwise=True, colwise=True)
        y, _ = temx.gemm(qh["q_row"], qh["s_row"], self.q_down["q_row"], self.q_down["s_row"])
        s = x + y
        out = temx.layernorm(s, *self.norm_out)
        return out["y"], (x, n, pre, qh, s, out["mu"], out["rsigma"])

    def backward(self, dout, saved):
        """Gradients of x, of the weights and of both norms' parameters."""
        x, n, pre, qh, s, mu, rsigma = saved
        d_out = temx.layernorm_backward(dout, s, self.norm_out[0], mu, rsigma)
        ds = d_out["dx"]
        q = temx.quantize(ds, rowwise=True, colwise=True)
        dh, _ = temx.gemm(q["q_row"], q["s_row"], self.q_down["q_col"], self.q_down["s_col"])
        dw_down, _ = temx.gemm(q["q_col"], q["s_col"], qh["q_col"], qh["s_col"])
        d = temx.gated_backward(dh, pre, activation=self.activation)
        dn, _ = temx.gemm(d["q_row"], d["s_row"], self.q_gate_up["q_col"], self.q_gate_up["s_col"])
        dw_gate_up, _ = temx.gemm(d["q_col"], d["s_col"], n["q_col"], n["s_col"])
        d_in = temx.layernorm_backward(dn, x, self.norm_in[0], n["mu"], n["rsigma"])
        return {"x": ds + d_in["dx"], "w_gate_up": dw_gate_up, "w_down": dw_down,
                "norm_in": (d_in["dgamma"], d_in["dbeta"]), "norm_out": (d_out["dgamma"], d_out["dbeta"])}

    def serve(self, x):
        """The forward pass alone, for any number of tokens."""
        n = temx.layernorm(x, *self.norm_in, stats=False)["y"]
        q = temx.quantize(n)
        h, _ = temx.gated_gemm(q["q_row"], q["s_row"], self.q_gate_up["q_row"], self.q_gate_up["s_row"],
                               activation=self.activation)
        q = temx.quantize(h)
        y, _ = temx.gemm(q["q_row"], q["s_row"], self.q_down["q_row"], self.q_down["s_row"])
        return temx.layernorm(x + y, *self.norm_out, stats=False)["y"]


def milliseconds(f, n=20):
    for _ in range(3):
        f()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    for _ in range(n):
        f()
    b.record()
    torch.cuda.synchronize()
    return a.elapsed_time(b) / n


def main():
    p = argparse.ArgumentParser()
    p.add_argument("--tokens", type=int, default=4096)
    p.add_argument("--hidden", type=int, default=1024)
    p.add_argument("--ffn", type=int, default=4096)
    p.add_argument("--activation", default="silu", choices=sorted(temx.ACTIVATIONS))
    a = p.parse_args()
    mlp = GatedMLP(a.hidden, a.ffn, a.activation)
    x = torch.randn(a.tokens, a.hidden, device="cuda").to(torch.bfloat16)
    dout = torch.randn_like(x)
    print(f"training, {a.tokens} tokens: {milliseconds(lambda: mlp.backward(dout, mlp.forward(x)[1])):.3f} ms a step")
    for tokens in (1, 64):
        print(f"serving, {tokens} tokens: {milliseconds(lambda: mlp.serve(x[:tokens])):.3f} ms")
    temx.te_mx_device_status()


if __name__ == "__main__":
    main()

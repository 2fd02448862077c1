"""A pre-norm mixture-of-experts block in MXFP8, trained and served.

    z   = x + residual,  n = RMSNorm(z)
    out = z + sum over a token's k experts of w_e W_out_e (act(W_gate_e n) * (W_up_e n))

with w the renormalised softmax of the router's logits n W_router^T.  A token is
quantised once and its codes go to the rows of its experts; the experts run in
grouped GEMMs; their outputs come back weighted and added to z.

    python examples/moe_block.py [--tokens 4096 --hidden 1024 --ffn 512 --experts 32 --k 4]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mxfp8_block_scaled_quantize_gb300 as temx  # noqa: E402


class MoEBlock:
    def __init__(self, hidden: int, ffn: int, experts: int, k: int, activation: str = "silu", seed: int = 0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        bf = torch.bfloat16
        self.hidden, self.ffn, self.experts, self.k, self.activation = hidden, ffn, experts, k, activation
        self.gamma = (1 + 0.1 * randn(hidden)).to(bf)
        self.w_router = (randn(experts, hidden) * hidden ** -0.5).to(bf)
        self.w_in = (randn(experts, 2 * ffn, hidden) * hidden ** -0.5).to(bf)        # gate rows, then up rows
        self.w_out = (randn(experts, hidden, ffn) * ffn ** -0.5).to(bf)
        # the weights and their transposes, quantised once per optimiser step
        self.q_in, self.q_in_t = self._quantised(self.w_in), self._quantised(self.w_in.transpose(1, 2))
        self.q_out, self.q_out_t = self._quantised(self.w_out), self._quantised(self.w_out.transpose(1, 2))

    @staticmethod
    def _quantised(w):
        q = temx.quantize(w.reshape(-1, w.shape[2]).contiguous())
        return q["q_row"].view(w.shape), q["s_row"]

    def _experts_of(self, n):
        """Router and plan for the normalised tokens n: (route, sort)."""
        r = temx.route(n @ self.w_router.t(), self.k)
        return r, temx.moe_sort(r["index"], self.experts)

    def forward(self, x, residual):
        """x, residual bf16 [tokens, hidden] -> (out, what the backward pass needs)."""
        n = temx.rmsnorm_quantize(x, self.gamma, residual=residual, dense=True)
        r, s = self._experts_of(n["y"])
        q, sc = temx.moe_dispatch(n["q_row"], s["row"], scales=n["s_row"])
        h, pre = temx.grouped_gated_gemm(s["group_m"], q, sc, *self.q_in, activation=self.activation, aux=True)
        qh = temx.quantize(h)
        y, _ = temx.grouped_gemm(s["group_m"], qh["q_row"], qh["s_row"], *self.q_out)
        out = temx.moe_combine(y, s["row"], weight=r["weight"], residual=n["z"])
        return out, (n, r, s, h, pre, y)

    def backward(self, dout, saved):
        """Gradients of x (and of the residual alike) and of the parameters."""
        n, r, s, h, pre, y = saved
        group_m, row, total = s["group_m"], s["row"], y.shape[0]
        d = temx.moe_combine_backward(dout, y, row, r["weight"])
        q = temx.quantize(d["dy"])
        dh, _ = temx.grouped_gemm(group_m, q["q_row"], q["s_row"], *self.q_out_t)
        columns = lambda t: temx.quantize_colwise_grouped(t, group_m)  # noqa: E731
        dw_out = temx.grouped_gemm_wgrad(group_m, total, columns(d["dy"]), columns(h))
        g = temx.gated_backward(dh, pre, activation=self.activation, dense=True, colwise=False)
        dx_rows, _ = temx.grouped_gemm(group_m, g["q_row"], g["s_row"], *self.q_in_t)
        dw_in = temx.grouped_gemm_wgrad(group_m, total, columns(g["d_gate_up"]), columns(temx.moe_dispatch(n["y"], row)))
        dlogits = temx.route_backward(d["dweight"], n["y"] @ self.w_router.t(), r["index"])
        # the gradient of dispatch is a combine without weights; the router's is added to it
        dn = temx.moe_combine(dx_rows, row, residual=dlogits @ self.w_router)
        b = temx.rmsnorm_backward(dn, n["z"], self.gamma, n["rsigma"], dz=dout)
        return {"x": b["dx"], "gamma": b["dgamma"], "w_router": dlogits.t() @ n["y"], "w_in": dw_in, "w_out": dw_out}

    def serve(self, x, residual):
        """The forward pass alone, for any number of tokens."""
        n = temx.rmsnorm_quantize(x, self.gamma, residual=residual, dense=True)
        r, s = self._experts_of(n["y"])
        q, sc = temx.moe_dispatch(n["q_row"], s["row"], scales=n["s_row"])
        h, _ = temx.grouped_gated_gemm(s["group_m"], q, sc, *self.q_in, activation=self.activation)
        qh = temx.quantize(h)
        y, _ = temx.grouped_gemm(s["group_m"], qh["q_row"], qh["s_row"], *self.q_out)
        return temx.moe_combine(y, s["row"], weight=r["weight"], residual=n["z"])


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
    p.add_argument("--ffn", type=int, default=512)
    p.add_argument("--experts", type=int, default=32)
    p.add_argument("--k", type=int, default=4)
    p.add_argument("--activation", default="silu", choices=sorted(temx.ACTIVATIONS))
    a = p.parse_args()
    block = MoEBlock(a.hidden, a.ffn, a.experts, a.k, a.activation)
    x, residual, dout = (torch.randn(a.tokens, a.hidden, device="cuda").to(torch.bfloat16) for _ in range(3))
    step = milliseconds(lambda: block.backward(dout, block.forward(x, residual)[1]))
    print(f"training, {a.tokens} tokens: {step:.3f} ms a step")
    for tokens in (1, 64):
        print(f"serving, {tokens} tokens: {milliseconds(lambda: block.serve(x[:tokens], residual[:tokens])):.3f} ms")
    temx.te_mx_device_status()


if __name__ == "__main__":
    main()

"""The example's block: its outputs and gradients against the same block in
float64 torch autograd on the unquantised weights.  Every operand of a GEMM is
rounded to E4M3 (half a step 2^-4, a uniform error within it 2^-4 / sqrt(3) of
the value at most in the mean square, near 0.026 over a binade), two operands a
product and up to four products in a chain, so relative 2-norm errors of up to
about 0.026 * sqrt(8) = 0.08 are the format's own; twice that bounds them."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BOUND = 0.16


def reference(mlp, x, dout):
    leaves = [t.double().requires_grad_() for t in (x, mlp.w_gate_up, mlp.w_down, *mlp.norm_in, *mlp.norm_out)]
    x, wg, wd, g1, b1, g2, b2 = leaves
    n = torch.nn.functional.layer_norm(x, x.shape[1:], g1, b1, 1e-5)
    g, u = (n @ wg.t()).chunk(2, dim=1)
    a = {"silu": torch.nn.functional.silu, "relu": torch.relu,
         "gelu": lambda t: torch.nn.functional.gelu(t, approximate="tanh")}[mlp.activation](g)
    out = torch.nn.functional.layer_norm(x + (a * u) @ wd.t(), x.shape[1:], g2, b2, 1e-5)
    out.backward(dout.double())
    return out.detach(), [t.grad for t in leaves]


def off(got, want):
    return ((got.double() - want).norm() / want.norm()).item()


@pytest.mark.parametrize("activation", ["silu", "gelu", "relu"])
def test_training_step(activation):
    from examples.gated_mlp import GatedMLP
    mlp = GatedMLP(512, 1024, activation, seed=1)
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(384, 512, generator=gen, device="cuda").to(torch.bfloat16)
    dout = torch.randn(384, 512, generator=gen, device="cuda").to(torch.bfloat16)
    out, saved = mlp.forward(x)
    grads = mlp.backward(dout, saved)
    want, wg = reference(mlp, x, dout)
    assert off(out, want) < BOUND
    for got, w, name in zip((grads["x"], grads["w_gate_up"], grads["w_down"], *grads["norm_in"], *grads["norm_out"]), wg,
                            ("x", "w_gate_up", "w_down", "gamma_in", "beta_in", "gamma_out", "beta_out")):
        assert off(got, w) < BOUND, name


@pytest.mark.parametrize("tokens", [1, 7, 130])
def test_serving_agrees_with_training(tokens):
    from examples.gated_mlp import GatedMLP
    mlp = GatedMLP(512, 2048, seed=3)
    x = torch.randn(tokens, 512, generator=torch.Generator(device="cuda").manual_seed(4), device="cuda").to(torch.bfloat16)
    want, _ = reference(mlp, x, torch.zeros_like(x))
    assert off(mlp.serve(x), want) < BOUND

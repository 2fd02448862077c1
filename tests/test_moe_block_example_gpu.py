"""The example's block: its outputs and gradients against the same block in float64
torch autograd on the unquantised weights, with the choices that the block made.
Every operand of a GEMM is rounded to E4M3 (half a step 2^-4, a uniform error within
it 2^-4 / sqrt(3) of the value at most in the mean square, near 0.026 over a binade),
two operands a product and up to four products in a chain, so relative 2-norm errors of
up to about 0.026 * sqrt(8) = 0.08 are the format's own; twice that bounds them.  The
router's gradients pass through differences of the weights' (g - sum w g), which keep
the errors of their terms: up to twice the share again."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BOUND = 0.16


def reference(block, x, residual, dout, index):
    leaves = [t.double().requires_grad_() for t in (x, residual, block.gamma, block.w_router, block.w_in, block.w_out)]
    x, residual, gamma, wr, wi, wo = leaves
    z = x + residual
    n = z * torch.rsqrt((z * z).mean(1, keepdim=True) + 1e-5) * gamma
    p = torch.softmax(n @ wr.t(), 1).gather(1, index.long())
    w = p / p.sum(1, keepdim=True)
    act = {"silu": torch.nn.functional.silu, "relu": torch.relu,
           "gelu": lambda t: torch.nn.functional.gelu(t, approximate="tanh")}[block.activation]
    out = z
    for e in range(block.experts):
        t, j = (index == e).nonzero(as_tuple=True)
        g, u = (n[t] @ wi[e].t()).chunk(2, dim=1)
        out = out.index_add(0, t, w[t, j, None] * ((act(g) * u) @ wo[e].t()))
    out.backward(dout.double())
    return out.detach(), dict(zip(("x", "residual", "gamma", "w_router", "w_in", "w_out"), (t.grad for t in leaves)))


def off(got, want):
    return ((got.double() - want).norm() / want.norm()).item()


@pytest.mark.parametrize("activation,tokens", [("silu", 300), ("gelu", 128), ("relu", 517)])
def test_training_step(activation, tokens):
    from examples.moe_block import MoEBlock
    block = MoEBlock(256, 128, 8, 2, activation, seed=1)
    gen = torch.Generator(device="cuda").manual_seed(2)
    x, residual, dout = (torch.randn(tokens, 256, generator=gen, device="cuda").to(torch.bfloat16) for _ in range(3))
    out, saved = block.forward(x, residual)
    grads = block.backward(dout, saved)
    want, wg = reference(block, x, residual, dout, saved[1]["index"])
    assert off(out, want) < BOUND
    assert torch.equal(wg["x"], wg["residual"])
    for name in ("x", "gamma", "w_in", "w_out"):
        assert off(grads[name], wg[name]) < BOUND, name
    assert off(grads["w_router"], wg["w_router"]) < 2 * BOUND


@pytest.mark.parametrize("tokens", [1, 7, 130])
def test_serving_agrees_with_training(tokens):
    from examples.moe_block import MoEBlock
    block = MoEBlock(512, 256, 16, 4, seed=3)
    gen = torch.Generator(device="cuda").manual_seed(4)
    x, residual = (torch.randn(tokens, 512, generator=gen, device="cuda").to(torch.bfloat16) for _ in range(2))
    out, saved = block.forward(x, residual)
    served = block.serve(x, residual)
    assert torch.equal(served, out)
    assert off(served, reference(block, x, residual, torch.zeros_like(x), saved[1]["index"])[0]) < BOUND

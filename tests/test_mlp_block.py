"""GPU: the example block (layer norm, two linear operators, their gradients)
against binary64 differentiation, its training, and its serving form."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location(
        "mlp_block", os.path.join(ROOT, "examples", "mlp_block.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def reference(block, x, delta):
    """out in binary64 with gradients, from the block's own weights."""
    p = [v.detach().double().cpu().requires_grad_() for v in block.parameters()]
    x = x.double().cpu().requires_grad_()
    gamma, beta, w1, b1, w2, bb2 = p
    s = x + delta.double().cpu()
    n = torch.nn.functional.layer_norm(s, (s.shape[-1],), gamma, beta, 1e-5)
    out = s + torch.nn.functional.gelu(n @ w1.t() + b1) @ w2.t() + bb2
    return out, x, p


@pytest.mark.parametrize("dtype,tol", [(torch.float32, 1e-5), (torch.bfloat16, 2.0 ** -6)])
@pytest.mark.parametrize("rows,hidden,width", [(70, 128, 512), (33, 100, 260)])
def test_block_against_binary64(example, rows, hidden, width, dtype, tol):
    """The whole chain.  Its outputs pass four roundings of intermediate tensors
    (n, z or h, dz, dn) and one of their own, each 2^-8 at most in bfloat16:
    in the norm they stay below four half steps, 2^-6 (in float32 the sums of a
    few hundred terms dominate, below 1e-5)."""
    block = example.MLPBlock(hidden, width, dtype, seed=3)
    g = torch.Generator(device="cuda").manual_seed(4)
    x, delta, dout = (torch.randn(rows, hidden, generator=g, device="cuda").to(dtype)
                      for _ in range(3))
    out, kept = block.forward(x, delta)
    dx, grads = block.backward(dout, kept)
    ref, rx, rp = reference(block, x, delta)
    ref.backward(dout.double().cpu())

    def off(a, b):
        return float((a.double().cpu() - b).norm() / b.norm())
    assert off(out, ref.detach()) <= tol
    assert off(dx, rx.grad) <= tol
    for got, want in zip(grads, rp):
        assert off(got, want.grad) <= tol


def test_training_lowers_the_loss(example):
    block = example.MLPBlock(256, 1024, seed=5)
    losses = example.train(block, 1024, 25)
    assert sum(losses[-5:]) < 0.7 * sum(losses[:5])


def test_server_gives_the_training_forward(example):
    """Serving one token from a graph: within a bfloat16 step or two of the
    batch's row (the sums are split differently)."""
    block = example.MLPBlock(512, 2048, seed=6)
    g = torch.Generator(device="cuda").manual_seed(7)
    x, delta = (torch.randn(9, 512, generator=g, device="cuda").bfloat16() for _ in range(2))
    out, _ = block.forward(x, delta)
    server = example.Server(block)
    for i in (0, 4, 8):
        one = server(x[i:i + 1], delta[i:i + 1])
        diff = (one.float() - out[i:i + 1].float()).abs()
        assert bool((diff <= 2.0 ** -6 * (1 + out[i:i + 1].float().abs())).all())

"""GPU: the example decoder block (layer norm, linear, head norms with rotation, gated linear,
and their gradients, one after another as a model runs them) against binary64 differentiation,
its training and its serving form."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location(
        "decoder_block", os.path.join(ROOT, "examples", "decoder_block.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def reference(block, x, positions, mask):
    """out in binary64 with gradients, from the block's own weights."""
    p = [v.detach().double().cpu().requires_grad_() for v in block.parameters()]
    gamma1, gamma_q, gamma_k, wqkv, wo, gamma2, w13, w2 = p
    x = x.double().cpu().requires_grad_()
    f = torch.nn.functional

    def heads(t, gamma):
        t = t / torch.sqrt((t * t).mean(-1, keepdim=True) + 1e-6) * gamma
        angle = positions.cpu().double().unsqueeze(-1) * block.inv_freq.cpu()
        turn = torch.polar(torch.ones_like(angle), angle).unsqueeze(-2)
        a, b = t.chunk(2, -1)
        w = torch.complex(a, b) * turn
        return torch.cat((w.real, w.imag), -1)
    n1 = f.layer_norm(x, x.shape[-1:], gamma1, None, 1e-5)
    q, k, v = block._split(n1 @ wqkv.t())
    q, k = heads(q, gamma_q), heads(k, gamma_k)
    shared = block.heads // block.groups
    q, k, v = q.transpose(1, 2), *(t.transpose(1, 2).repeat_interleave(shared, 1) for t in (k, v))
    score = (q @ k.transpose(2, 3)) * block.size ** -0.5
    o = torch.softmax(score.masked_fill(~mask.cpu(), float("-inf")), -1) @ v
    s = x + o.transpose(1, 2).flatten(-2) @ wo.t()
    n2 = f.layer_norm(s, s.shape[-1:], gamma2, None, 1e-5)
    gate, up = (n2 @ w13.t()).chunk(2, -1)
    return s + (f.silu(gate) * up) @ w2.t(), x, p


@pytest.mark.parametrize("dtype,tol", [(torch.float32, 1e-5), (torch.bfloat16, 2.0 ** -5)])
@pytest.mark.parametrize("batch,seq,hidden,heads,groups,size,width",
                         [(2, 33, 128, 4, 2, 32, 256), (1, 50, 100, 3, 1, 20, 130)])
def test_block_against_binary64(example, batch, seq, hidden, heads, groups, size, width, dtype,
                                tol):
    """The whole chain.  A gradient passes at most eight roundings of intermediate tensors (n1,
    qkv, q or k, o, attn or S, n2, z or dz, h or dh and the like) and one of its own, each 2^-8
    at most in bfloat16: in the norm they stay below eight half steps, 2^-5 (in float32 the sums
    of a few hundred terms dominate, below 1e-5)."""
    block = example.DecoderBlock(hidden, heads, groups, size, width, dtype, seed=3)
    g = torch.Generator(device="cuda").manual_seed(4)
    for gamma in (block.gamma1, block.gamma_q, block.gamma_k, block.gamma2):
        gamma.copy_(1 + 0.2 * torch.randn(gamma.shape, generator=g, device="cuda"))
    x, dout = (torch.randn(batch, seq, hidden, generator=g, device="cuda").to(dtype)
               for _ in range(2))
    positions = torch.arange(1000, 1000 + seq, device="cuda")
    mask = example.causal(seq)
    out, kept = block.forward(x, positions, mask)
    dx, grads = block.backward(dout, kept)
    ref, rx, rp = reference(block, x, positions, mask)
    ref.backward(dout.double().cpu())

    def off(a, b):
        return float((a.double().cpu() - b).norm() / b.norm())
    assert off(out, ref.detach()) <= tol
    assert off(dx, rx.grad) <= tol
    for got, want in zip(grads, rp):
        assert off(got, want.grad) <= tol


def test_training_runs(example):
    block = example.DecoderBlock(128, 4, 2, 32, 256, seed=5)
    before = [p.clone() for p in block.parameters()]
    losses = example.train(block, 2, 64, 3)
    assert len(losses) == 3 and all(v == v and v < float("inf") for v in losses)
    assert all(bool((p != b).any()) for p, b in zip(block.parameters()[3:5], before[3:5]))


def test_server_gives_the_training_forward(example):
    """Tokens one at a time from a graph: the batch's rows, but for bfloat16 roundings turned
    (the sums are split differently; five tensors on the way, two steps of 2^-8 each)."""
    block = example.DecoderBlock(256, 4, 2, 64, 512, seed=6)
    g = torch.Generator(device="cuda").manual_seed(7)
    x = torch.randn(1, 20, 256, generator=g, device="cuda").bfloat16()
    out, _ = block.forward(x, torch.arange(20, device="cuda"), example.causal(20))
    server = example.Server(block, 20)
    for i in range(20):
        one = server(x[:, i:i + 1])
        off = float((one[:, 0].float() - out[:, i].float()).norm() / out[:, i].float().norm())
        assert off <= 10 * 2.0 ** -8, i
    with pytest.raises(ValueError, match="no room"):
        server(x[:, :1])

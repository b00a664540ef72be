"""A pre-norm MLP block on a residual stream, trained and served with the
framework's kernels:

    S = x + delta                          (delta: what the layer before adds)
    out = S + W2 gelu(W1 LayerNorm(S) + b1) + b2

    python examples/mlp_block.py [--rows 4096] [--hidden 1024] [--steps 30]

trains the block on a synthetic target with plain gradient descent, then serves
single tokens from a CUDA graph.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import residual_add_normalization_gb300 as b2  # noqa: E402

GELU = b2.ACTIVATIONS["gelu"]


class MLPBlock:
    """Weights of one block; ``width`` inner features."""

    def __init__(self, hidden, width, dtype=torch.bfloat16, device="cuda", seed=0):
        gen = torch.Generator(device=device).manual_seed(seed)

        def normal(*shape, scale):
            return (torch.randn(*shape, generator=gen, device=device) * scale).to(dtype)
        self.gamma = torch.ones(hidden, dtype=dtype, device=device)
        self.beta = torch.zeros(hidden, dtype=dtype, device=device)
        self.w1 = normal(width, hidden, scale=hidden ** -0.5)
        self.b1 = torch.zeros(width, dtype=dtype, device=device)
        self.w2 = normal(hidden, width, scale=width ** -0.5)
        self.b2 = torch.zeros(hidden, dtype=dtype, device=device)

    def parameters(self):
        return [self.gamma, self.beta, self.w1, self.b1, self.w2, self.b2]

    def forward(self, x, delta):
        """out, and what backward() needs."""
        n, s, mean, inv = b2.skip_layer_stats(x, delta, self.gamma, self.beta)
        h, z = b2.linear(n, self.w1, self.b1, activation=GELU, want_z=True)
        out, _ = b2.linear(h, self.w2, self.b2, residual=s)
        return out, (n, s, mean, inv, z, h)

    def serve(self, x, delta):
        """out alone: nothing is kept."""
        n, s = b2.skip_layer(x, delta, self.gamma, self.beta)
        h, _ = b2.linear(n, self.w1, self.b1, activation=GELU)
        return b2.linear(h, self.w2, self.b2, residual=s)[0]

    def backward(self, dout, kept):
        """Gradient of x (and of delta, the same), and of each parameter."""
        n, s, mean, inv, z, h = kept
        dh, dw2, db2 = b2.linear_grad(dout, h, self.w2)
        dn, dw1, db1 = b2.linear_grad(dh, n, self.w1, z, activation=GELU)
        # the stream carries dout past the block: it joins the norm's gradient there
        dx, dgamma, dbeta, _ = b2.skip_layer_grad(dn, s, mean, inv, self.gamma, ds=dout)
        return dx, [dgamma, dbeta, dw1, db1, dw2, db2]


def train(block, rows, steps, seed=1):
    """Losses of `steps` steps of gradient descent with momentum towards a fixed
    random map of the input; the weights' masters are float32."""
    hidden, device, dtype = block.gamma.numel(), block.gamma.device, block.gamma.dtype
    masters = [p.float() for p in block.parameters()]
    momenta = [torch.zeros_like(m) for m in masters]
    lr = 2.0 / block.w1.shape[0]
    gen = torch.Generator(device=device).manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=device)
    target = normal(hidden, hidden) * (0.5 * hidden ** -0.5)
    losses = []
    for _ in range(steps):
        x, delta = normal(rows, hidden), normal(rows, hidden)
        want = x + delta + torch.tanh(x + delta) @ target
        out, kept = block.forward(x.to(dtype), delta.to(dtype))
        err = out.float() - want
        losses.append(float(err.square().mean()))
        _, grads = block.backward((err * (2.0 / rows)).to(dtype), kept)
        for p, m, v, g in zip(block.parameters(), masters, momenta, grads):
            v.mul_(0.8).add_(g)
            m.sub_(v, alpha=lr)
            p.copy_(m)
    b2.linear_status()
    b2.rows_status()
    return losses


class Server:
    """One token at a time from a CUDA graph."""

    def __init__(self, block):
        self.x = torch.zeros(1, block.gamma.numel(), dtype=block.gamma.dtype,
                             device=block.gamma.device)
        self.delta = torch.zeros_like(self.x)
        block.serve(self.x, self.delta)  # loads the kernels before the capture
        torch.cuda.synchronize()
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self.out = block.serve(self.x, self.delta)

    def __call__(self, x, delta):
        self.x.copy_(x)
        self.delta.copy_(delta)
        self.graph.replay()
        return self.out.clone()


def main():
    ap = argparse.ArgumentParser(description=__doc__,
                                 formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--rows", type=int, default=4096)
    ap.add_argument("--hidden", type=int, default=1024)
    ap.add_argument("--steps", type=int, default=30)
    a = ap.parse_args()
    block = MLPBlock(a.hidden, 4 * a.hidden)
    losses = train(block, a.rows, a.steps)
    print("loss: first %.4f, last %.4f" % (losses[0], losses[-1]))
    server = Server(block)
    x, delta = (torch.randn(1, a.hidden, device="cuda").bfloat16() for _ in range(2))
    start, stop = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    server(x, delta)
    start.record()
    for _ in range(100):
        server.graph.replay()
    stop.record()
    stop.synchronize()
    print("one token: %.1f us" % (start.elapsed_time(stop) * 10))


if __name__ == "__main__":
    main()

"""A pre-norm decoder block on a residual stream, trained and served with the framework's
kernels (attention itself in plain torch operations):

    q, k, v = heads of Wqkv LayerNorm(x);  q, k = rotation(RMSNorm(q)), rotation(RMSNorm(k))
    S   = x + Wo attention(q, k, v)
    out = S + W2 (silu(Wg LayerNorm(S)) * (Wu LayerNorm(S)))

    python examples/decoder_block.py [--seq 512] [--hidden 512] [--steps 20]

trains the block on a synthetic target with plain gradient descent, then serves single
tokens from a CUDA graph that keeps the keys and values of the tokens before.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import residual_add_normalization_gb300 as b2  # noqa: E402

SILU = b2.ACTIVATIONS["silu"]


def attention(q, k, v, mask):
    """(batch, seq, heads, size) against (batch, length, groups, size); ``mask`` (seq, length)
    is where a query sees a key.  Heads share their group's keys; softmax in binary32."""
    shared = q.shape[2] // k.shape[2]
    qf, kf, vf = (t.float().transpose(1, 2) for t in (q, k, v))
    kf, vf = (t.repeat_interleave(shared, 1) for t in (kf, vf))
    score = (qf @ kf.transpose(2, 3)) * q.shape[-1] ** -0.5
    p = torch.softmax(score.masked_fill(~mask, float("-inf")), -1)
    return (p @ vf).transpose(1, 2).to(q.dtype)


class DecoderBlock:
    """Weights of one block: ``heads`` query heads of ``size`` in ``groups`` groups, ``width``
    inner features."""

    def __init__(self, hidden, heads, groups, size, width, dtype=torch.bfloat16, device="cuda",
                 seed=0):
        gen = torch.Generator(device=device).manual_seed(seed)

        def normal(rows, cols):
            return (torch.randn(rows, cols, generator=gen, device=device) * cols ** -0.5).to(dtype)

        def ones(n):
            return torch.ones(n, dtype=dtype, device=device)
        self.heads, self.groups, self.size = heads, groups, size
        self.gamma1, self.gamma2 = ones(hidden), ones(hidden)
        self.gamma_q, self.gamma_k = ones(size), ones(size)
        self.wqkv = normal((heads + 2 * groups) * size, hidden)
        self.wo = normal(hidden, heads * size)
        self.w13 = normal(2 * width, hidden)  # the gate's rows, then those of what it gates
        self.w2 = normal(hidden, width)
        self.inv_freq = b2.rotary_frequencies(size, device=device)

    def parameters(self):
        return [self.gamma1, self.gamma_q, self.gamma_k, self.wqkv, self.wo, self.gamma2, self.w13,
                self.w2]

    def _split(self, qkv):
        """Views of the queries, keys and values in the product's rows."""
        t = qkv.unflatten(-1, (self.heads + 2 * self.groups, self.size))
        return t.split([self.heads, self.groups, self.groups], -2)

    def _mlp(self, attn, x):
        n2, s, mean, inv = b2.skip_layer_stats(attn, x, self.gamma2)
        h, z = b2.gated_linear(n2, self.w13, activation=SILU, want_z=True)
        out, _ = b2.linear(h, self.w2, residual=s)
        return out, (n2, s, mean, inv, h, z)

    def forward(self, x, positions, mask):
        """out of x (batch, seq, hidden), and what backward() needs."""
        n1, _, mean, inv = b2.skip_layer_stats(x, None, self.gamma1)
        qkv, _ = b2.linear(n1, self.wqkv)
        q0, k0, v = self._split(qkv)
        q, k = b2.head_rms_rotary(q0, k0, self.gamma_q, self.gamma_k, positions, self.inv_freq)
        with torch.enable_grad():
            leaves = [t.detach().requires_grad_() for t in (q, k, v)]
            o = attention(*leaves, mask)
        oc = o.detach().flatten(-2).contiguous()
        attn, _ = b2.linear(oc, self.wo)
        out, mlp = self._mlp(attn, x)
        return out, (x, n1, mean, inv, q0, k0, leaves, o, oc, positions, mlp)

    def backward(self, dout, kept):
        """Gradient of x, and of each parameter."""
        x, n1, mean, inv, q0, k0, leaves, o, oc, positions, (n2, s, mean2, inv2, h, z) = kept
        dh, dw2, _ = b2.linear_grad(dout, h, self.w2, want_bias=False)
        dn2, dw13, _ = b2.gated_linear_grad(dh, n2, self.w13, z, activation=SILU, want_bias=False)
        # the stream carries dout past the MLP, and ds past the attention
        ds, dgamma2, _, _ = b2.skip_layer_grad(dn2, s, mean2, inv2, self.gamma2, ds=dout,
                                               want_beta=False)
        do, dwo, _ = b2.linear_grad(ds, oc, self.wo, want_bias=False)
        dq, dk, dv = torch.autograd.grad(o, leaves, do.view(o.shape))
        # of the product's rows: queries' and keys' gradients are stored in their places
        dqkv = torch.empty(x.shape[:-1] + (self.wqkv.shape[0],), dtype=x.dtype, device=x.device)
        dq0, dk0, dv0 = self._split(dqkv)
        dv0.copy_(dv)
        _, _, dgamma_q, dgamma_k = b2.head_rms_rotary_grad(
            dq, dk, q0, k0, self.gamma_q, self.gamma_k, positions, self.inv_freq, dq_out=dq0,
            dk_out=dk0)
        dn1, dwqkv, _ = b2.linear_grad(dqkv, n1, self.wqkv, want_bias=False)
        dx, dgamma1, _, _ = b2.skip_layer_grad(dn1, x, mean, inv, self.gamma1, ds=ds,
                                               want_beta=False)
        return dx, [dgamma1, dgamma_q, dgamma_k, dwqkv, dwo, dgamma2, dw13, dw2]

    def serve(self, x, positions, keys, values):
        """out of one token per sequence, x (batch, 1, hidden), at ``positions`` (1,); its keys
        and values join those of the tokens before (batch, length, groups, size)."""
        n1, _ = b2.skip_layer(x, None, self.gamma1)
        qkv, _ = b2.linear(n1, self.wqkv)
        q0, k0, v = self._split(qkv)
        q, k = b2.head_rms_rotary(q0, k0, self.gamma_q, self.gamma_k, positions, self.inv_freq)
        keys.index_copy_(1, positions, k)
        values.index_copy_(1, positions, v)
        mask = torch.arange(keys.shape[1], device=x.device) <= positions
        o = attention(q, keys, values, mask.view(1, -1))
        attn, _ = b2.linear(o.flatten(-2).contiguous(), self.wo)
        n2, s = b2.skip_layer(attn, x, self.gamma2)
        h, _ = b2.gated_linear(n2, self.w13, activation=SILU)
        return b2.linear(h, self.w2, residual=s)[0]


def causal(seq, device="cuda"):
    return torch.ones(seq, seq, dtype=torch.bool, device=device).tril()


def train(block, batch, seq, steps, seed=1):
    """Losses of `steps` steps of gradient descent towards a fixed random map of the token
    before; the weights' masters are float32."""
    hidden, device, dtype = block.gamma1.numel(), block.gamma1.device, block.gamma1.dtype
    masters = [p.float() for p in block.parameters()]
    gen = torch.Generator(device=device).manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=device)
    target = normal(hidden, hidden) * (0.5 * hidden ** -0.5)
    positions, mask = torch.arange(seq, device=device), causal(seq, device)
    losses = []
    for _ in range(steps):
        x = normal(batch, seq, hidden)
        want = x + torch.tanh(torch.roll(x, 1, 1) @ target)
        out, kept = block.forward(x.to(dtype), positions, mask)
        err = out.float() - want
        losses.append(float(err.square().mean()))
        _, grads = block.backward((err * (2.0 / (batch * seq))).to(dtype), kept)
        for p, m, g in zip(block.parameters(), masters, grads):
            m.sub_(g, alpha=2.0 / hidden)
            p.copy_(m)
    b2.linear_status()
    b2.rows_status()
    return losses


class Server:
    """One token at a time from a CUDA graph, at most ``length`` of them."""

    def __init__(self, block, length, batch=1):
        device, dtype = block.gamma1.device, block.gamma1.dtype
        self.x = torch.zeros(batch, 1, block.gamma1.numel(), dtype=dtype, device=device)
        self.position = torch.zeros(1, dtype=torch.int64, device=device)
        self.keys, self.values = (torch.zeros(batch, length, block.groups, block.size, dtype=dtype,
                                              device=device) for _ in range(2))
        block.serve(self.x, self.position, self.keys, self.values)  # loads the kernels
        torch.cuda.synchronize()
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self.out = block.serve(self.x, self.position, self.keys, self.values)
        self.length, self.next = length, 0

    def __call__(self, x):
        if self.next == self.length:
            raise ValueError(f"no room for more than {self.length} tokens")
        self.x.copy_(x)
        self.position.fill_(self.next)
        self.next += 1
        self.graph.replay()
        return self.out.clone()


def main():
    ap = argparse.ArgumentParser(description=__doc__,
                                 formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--seq", type=int, default=512)
    ap.add_argument("--hidden", type=int, default=512)
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args()
    block = DecoderBlock(a.hidden, a.hidden // 64, max(1, a.hidden // 256), 64, 2 * a.hidden)
    losses = train(block, 4, a.seq, a.steps)
    print("loss: first %.4f, last %.4f" % (losses[0], losses[-1]))
    server = Server(block, a.seq)
    x = torch.randn(1, 1, a.hidden, device="cuda").bfloat16()
    start, stop = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    server(x)
    start.record()
    for _ in range(100):
        server.graph.replay()
    stop.record()
    stop.synchronize()
    print("one token: %.1f us" % (start.elapsed_time(stop) * 10))


if __name__ == "__main__":
    main()

"""What is measured of the operators around attention and of the gated MLP.

With layer normalization and the linear operator these make a pre-norm decoder
block on a residual stream, in training and in serving:

  rotary       rotation of query and key heads by their position: pairs (a, b) of
               a head become (a c - b s, b c + a s), c and s the scaled cosine and
               sine of position * frequency; or the inverse rotation (its gradient)
  heads        the same after an RMS norm of each head, x / sqrt(mean(x^2) + eps) * gamma
  heads_grad   its gradients: of queries, keys and both gammas
  gated        act(x Wg^T + bg) * (x Wu^T + bu), with both products kept for training
  gated_grad   its gradients: of x, of the weights (gate rows, then up rows), of the biases

`own` chooses between the framework's kernels and the plain form in torch
operations.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
EPS = 1e-6
ACTIVATIONS = {"none": 0, "silu": 1, "gelu": 2, "gelu_tanh": 3, "relu": 4}

# Work of the largest listed cases: a batch of 8 x 2048 tokens.
LARGEST_ELEMENTS = 16384 * 40 * 128
LARGEST_MACS = 2 * 16384 * 4096 * 16384


def _heads(name, op, batch, seq, q, k, size, rot, layout, t, m, *, packed=True, start=0, factor=1.0,
           inverse=False):
    return {"name": name, "op": op, "batch": batch, "seq": seq, "q": q, "k": k, "size": size,
            "rot": rot, "layout": layout, "t": t, "m": m, "packed": packed, "start": start,
            "factor": factor, "inverse": inverse}


def _gated(name, op, rows, n_in, n_out, t, act, bias, keep):
    return {"name": name, "op": op, "rows": rows, "in": n_in, "out": n_out, "t": t, "act": act,
            "bias": bias, "keep": keep}


def listed():
    return [
        # serving: one new token far into a scaled context, its heads next to one another in
        # the product's row
        _heads("heads_decode_bf16_1x40x128", "heads", 1, 1, 32, 8, 128, 128, "half", "bf16",
               "bf16", start=100000, factor=8.0),
        # ragged token count, odd numbers of heads, part of the head rotated; float32 weights
        _heads("heads_odd_fp16_7x111x6x80", "heads", 7, 111, 5, 1, 80, 40, "interleaved", "f16",
               "f32", start=11),
        # training or prefill over 8 x 2048 tokens
        _heads("heads_bf16_8x2048x40x128", "heads", 8, 2048, 32, 8, 128, 128, "half", "bf16",
               "bf16"),
        # a small float32 model's training step (8 sequences of 64, 12 heads each)
        _heads("heads_grad_fp32_8x64x24x64", "heads_grad", 8, 64, 12, 12, 64, 64, "half", "f32",
               "f32", packed=False),
        # training over 8 x 2048 tokens
        _heads("heads_grad_bf16_8x2048x40x128", "heads_grad", 8, 2048, 32, 8, 128, 128, "half",
               "bf16", "bf16"),
        # serving 64 sequences, a token each, all at places of their own
        _heads("rotary_decode_fp16_64x40x128", "rotary", 64, 1, 32, 8, 128, 64, "interleaved",
               "f16", "f16", start=30000),
        # the gradient of a float32 model's rotation over a long sequence of an odd length
        _heads("rotary_inverse_fp32_1x8191x32x96", "rotary", 1, 8191, 16, 16, 96, 96, "half",
               "f32", "f32", factor=4.0, inverse=True),
        # serving: one token through the gated product that widens the stream
        _gated("gated_decode_bf16_1x4096x8192", "gated", 1, 4096, 8192, "bf16", "silu", False,
               False),
        # sizes that fit neither a tile nor a 16-byte row
        _gated("gated_odd_fp16_777x1027x1283", "gated", 777, 1027, 1283, "f16", "gelu_tanh", True,
               True),
        # training or prefill over 8 x 2048 tokens
        _gated("gated_bf16_16384x4096x8192", "gated", 16384, 4096, 8192, "bf16", "silu", False,
               True),
        # a small float32 model's training step (8 sequences of 64)
        _gated("gated_grad_fp32_512x768x768", "gated_grad", 512, 768, 768, "f32", "silu", True,
               True),
        # training over 8 x 2048 tokens (the largest case)
        _gated("gated_grad_bf16_16384x4096x8192", "gated_grad", 16384, 4096, 8192, "bf16", "silu",
               False, True),
    ]


def _spread(rng, lo, hi, step=64):
    """A whole number spread over the logarithm of [lo, hi]; two in three are multiples of `step`."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    if v >= step and rng.random() < 2 / 3:
        return min(hi, max(step, int(v) // step * step))
    return min(hi, max(lo, int(v)))


def draw(rng):
    op = rng.choice(["rotary", "heads", "heads_grad", "gated", "gated_grad"])
    t = rng.choice(["bf16", "f16", "f32"])
    if op in ("rotary", "heads", "heads_grad"):
        while True:
            batch, seq = _spread(rng, 1, 64, 8), _spread(rng, 1, 16384)
            q = _spread(rng, 1, 64, 8)
            k = rng.choice([1, q, max(1, q // 4), max(1, q // 8)])
            size = _spread(rng, 16, 256, 32)
            if batch * seq * (q + k) * size <= LARGEST_ELEMENTS // (2 if t == "f32" else 1):
                break
        rot = rng.choice([size, size // 2, size // 4]) // 2 * 2
        case = _heads("", op, batch, seq, q, k, size, max(2, rot),
                      rng.choice(["half", "interleaved"]), t, rng.choice([t, "f32"]),
                      packed=rng.random() < 0.7, start=rng.choice([0, _spread(rng, 1, 1000000)]),
                      factor=rng.choice([1.0, 4.0, 32.0]),
                      inverse=op == "rotary" and rng.random() < 0.5)
    else:
        most = LARGEST_MACS // (32 if t == "f32" else 4)
        while True:
            rows = _spread(rng, 1, 16384)
            n_in, n_out = _spread(rng, 64, 16384), _spread(rng, 64, 8192)
            if 2 * rows * n_in * n_out <= most:
                break
        act = rng.choice(sorted(ACTIVATIONS))
        case = _gated("", op, rows, n_in, n_out, t, act, rng.random() < 0.5,
                      op == "gated_grad" or rng.random() < 0.5)
    del case["name"]
    return case


class _Maker:
    """Random tensors from one seed, on the GPU."""

    def __init__(self, seed):
        self.gen = torch.Generator(device="cuda")
        self.gen.manual_seed(seed)

    def normal(self, shape, t, scale=1.0, mean=0.0):
        v = torch.randn(shape, generator=self.gen, device="cuda", dtype=torch.float32)
        return v.mul_(scale).add_(mean).to(DTYPES[t])


def _frequencies(rot, factor):
    """Radians a position, binary64, of a context `factor` times as long as the original one of
    8192: pairs that turn less than once over it are slowed down by the factor, those that turn
    more than 32 times are not, the others in proportion."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    if factor != 1.0:
        keep = ((8192 * f / (2 * math.pi) - 1.0) / 31.0).clamp(0.0, 1.0)
        f = f * keep + f / factor * (1.0 - keep)
    return f


def prepare(case, seed):
    mk = _Maker(seed)
    st = {"case": case}
    op, t = case["op"], case["t"]
    if op in ("rotary", "heads", "heads_grad"):
        batch, seq, nq, nk, d = (case[n] for n in ("batch", "seq", "q", "k", "size"))
        if case["packed"]:  # queries, keys and values next to one another, as a product leaves them
            rows = mk.normal((batch, seq, nq + 2 * nk, d), t, 2.0)
            st["q"], st["k"] = rows[:, :, :nq], rows[:, :, nq:nq + nk]
        else:
            st["q"], st["k"] = (mk.normal((batch, seq, n, d), t, 2.0) for n in (nq, nk))
        first = torch.randint(0, case["start"] + 1, (batch, 1), generator=mk.gen, device="cuda")
        st["positions"] = first + torch.arange(seq, device="cuda")
        st["inv_freq"] = _frequencies(case["rot"], case["factor"]).cuda()
        st["scale"] = 0.1 * math.log(case["factor"]) + 1.0
        if op != "rotary":
            st["gamma_q"], st["gamma_k"] = (mk.normal((d,), case["m"], 0.1, 1.0) for _ in range(2))
        if op == "heads_grad":
            st["dq"], st["dk"] = (mk.normal((batch, seq, n, d), t, 0.1) for n in (nq, nk))
        return st
    rows, n_in, n_out = case["rows"], case["in"], case["out"]
    st["x"] = mk.normal((rows, n_in), t)
    st["w"] = mk.normal((2 * n_out, n_in), t, 1.0 / math.sqrt(n_in))
    if op == "gated":
        st["bias"] = mk.normal((2 * n_out,), t, 0.1) if case["bias"] else None
    else:
        st["dh"] = mk.normal((rows, n_out), t, 0.1)
        st["z"] = mk.normal((rows, 2 * n_out), t)
    return st


# -- the plain form: binary32, one rounding at the end ------------------------

def _angles(st):
    """Scaled cosine and sine, (batch, seq, 1, rot / 2) in binary32; the angles in binary64."""
    angle = st["positions"].double().unsqueeze(-1) * st["inv_freq"]
    return ((f(angle) * st["scale"]).float().unsqueeze(2) for f in (torch.cos, torch.sin))


def _rotate(case, v, cos, sin):
    rot = case["rot"]
    out = torch.empty_like(v)
    out[..., rot:] = v[..., rot:]
    if case["layout"] == "half":
        a, b = v[..., :rot // 2], v[..., rot // 2:rot]
        out[..., :rot // 2], out[..., rot // 2:rot] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = v[..., 0:rot:2], v[..., 1:rot:2]
        out[..., 0:rot:2], out[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
    return out


def _act(z, name):
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    if name == "relu":
        return torch.clamp(z, min=0.0)
    return z


def _act_slope(z, name):
    if name == "silu":
        s = torch.sigmoid(z)
        return s * (1.0 + z * (1.0 - s))
    if name == "gelu":
        return (0.5 * (1.0 + torch.erf(z * math.sqrt(0.5)))
                + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi)))
    if name == "gelu_tanh":
        k = math.sqrt(2.0 / math.pi)
        th = torch.tanh(k * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + th) + 0.5 * z * (1.0 - th * th) * k * (1.0 + 3 * 0.044715 * z * z)
    if name == "relu":
        return (z > 0).to(z.dtype)
    return torch.ones_like(z)


def _plain(st):
    case = st["case"]
    op, t = case["op"], DTYPES[case["t"]]
    if op == "rotary":
        cos, sin = _angles(st)
        sin = -sin if case["inverse"] else sin
        return {n: _rotate(case, st[n].float(), cos, sin).to(t) for n in ("q", "k")}
    if op == "heads":
        cos, sin = _angles(st)
        out = {}
        for n in ("q", "k"):
            x = st[n].float()
            inv = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
            out[n] = _rotate(case, x * inv * st["gamma_" + n].float(), cos, sin).to(t)
        return out
    if op == "heads_grad":
        cos, sin = _angles(st)
        out = {}
        for n in ("q", "k"):
            x = st[n].float()
            inv = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
            u = x * inv
            da = _rotate(case, st["d" + n].float(), cos, -sin)
            g = da * st["gamma_" + n].float()
            out["d" + n] = (inv * (g - u * (g * u).mean(-1, keepdim=True))).to(t)
            out["dgamma_" + n] = (da * u).flatten(0, 2).sum(0).to(DTYPES[case["m"]])
        return out
    n, act = case["out"], case["act"]
    x, w = st["x"].float(), st["w"].float()
    if op == "gated":
        z = x @ w.t()
        if st["bias"] is not None:
            z = z + st["bias"].float()
        out = {"h": (_act(z[:, :n], act) * z[:, n:]).to(t)}
        if case["keep"]:
            out["z"] = z.to(t)
        return out
    dh, z = st["dh"].float(), st["z"].float()
    gate, up = z[:, :n], z[:, n:]
    dz = torch.cat((dh * up * _act_slope(gate, act), dh * _act(gate, act)), 1)
    out = {"dx": (dz @ w).to(t), "dw": (dz.t() @ x).to(t)}
    if case["bias"]:
        out["db"] = dz.sum(0).to(t)
    return out


# -- the framework's kernels --------------------------------------------------

def _own(st):
    import residual_add_normalization_gb300 as b2
    case = st["case"]
    op = case["op"]
    if op in ("rotary", "heads", "heads_grad"):
        interleaved = case["layout"] == "interleaved"
        if op == "rotary":
            q, k = b2.rotary(st["q"], st["k"], st["positions"], st["inv_freq"],
                             interleaved=interleaved, scale=st["scale"], inverse=case["inverse"])
            return {"q": q, "k": k}
        if op == "heads":
            q, k = b2.head_rms_rotary(st["q"], st["k"], st["gamma_q"], st["gamma_k"],
                                      st["positions"], st["inv_freq"], epsilon=EPS,
                                      interleaved=interleaved, scale=st["scale"])
            return {"q": q, "k": k}
        dq, dk, dgamma_q, dgamma_k = b2.head_rms_rotary_grad(
            st["dq"], st["dk"], st["q"], st["k"], st["gamma_q"], st["gamma_k"], st["positions"],
            st["inv_freq"], epsilon=EPS, interleaved=interleaved, scale=st["scale"])
        return {"dq": dq, "dgamma_q": dgamma_q, "dk": dk, "dgamma_k": dgamma_k}
    act = ACTIVATIONS[case["act"]]
    if op == "gated":
        h, z = b2.gated_linear(st["x"], st["w"], st["bias"], activation=act, want_z=case["keep"])
        return {"h": h, "z": z} if case["keep"] else {"h": h}
    dx, dw, db = b2.gated_linear_grad(st["dh"], st["x"], st["w"], st["z"], activation=act,
                                      want_bias=case["bias"])
    return {"dx": dx, "dw": dw, "db": db} if case["bias"] else {"dx": dx, "dw": dw}


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    es, op = SIZE[case["t"]], case["op"]
    if op in ("rotary", "heads", "heads_grad"):
        tokens = case["batch"] * case["seq"]
        n = tokens * (case["q"] + case["k"]) * case["size"]
        extra = 8 * tokens + 4 * case["rot"]
        if op != "rotary":
            extra += (2 if op == "heads" else 4) * case["size"] * SIZE[case["m"]]
        tensors, per = {"rotary": (2, 3), "heads": (2, 7), "heads_grad": (3, 14)}[op]
        return {"bytes": tensors * n * es + extra, "flops": per * n}
    rows, n_in, n_out = case["rows"], case["in"], case["out"]
    if op == "gated":
        n = (rows * n_in + 2 * n_in * n_out + case["bias"] * 2 * n_out
             + rows * n_out * (1 + 2 * case["keep"]))
        return {"bytes": n * es, "flops": 4 * rows * n_in * n_out}
    n = 2 * (rows * n_in + 2 * n_in * n_out) + case["bias"] * 2 * n_out + 3 * rows * n_out
    return {"bytes": n * es, "flops": 8 * rows * n_in * n_out}


# -- the definitions in 64 bits -----------------------------------------------

def _turned64(case, v, turn):
    """v with its pairs, as complex numbers, multiplied by `turn`."""
    rot, h = case["rot"], case["rot"] // 2
    if case["layout"] == "half":
        w = torch.complex(v[..., :h].contiguous(), v[..., h:rot].contiguous()) * turn
        return torch.cat((w.real, w.imag, v[..., rot:]), -1)
    w = torch.view_as_complex(v[..., :rot].reshape(v.shape[:-1] + (h, 2)).contiguous()) * turn
    return torch.cat((torch.view_as_real(w).flatten(-2), v[..., rot:]), -1)


def _sigmoid64(z):
    return 1.0 / (1.0 + torch.exp(-z))


def _cdf64(z):
    """The normal distribution's cumulative function (no cancellation in its tail)."""
    return 0.5 * torch.special.erfc(-z / math.sqrt(2.0))


def _tanh_gate64(z):
    """(1 + tanh(u)) / 2 = sigmoid(2 u) for u = sqrt(2/pi) (z + 0.044715 z^3)."""
    return _sigmoid64(2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3))


def _value64(z, name):
    if name == "silu":
        return z * _sigmoid64(z)
    if name == "gelu":
        return z * _cdf64(z)
    if name == "gelu_tanh":
        return z * _tanh_gate64(z)
    if name == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    return z


def _derivative64(z, name):
    if name == "silu":
        s = _sigmoid64(z)
        return s + z * s * (1.0 - s)
    if name == "gelu":
        return _cdf64(z) + z * torch.exp(-z * z / 2.0) / math.sqrt(2.0 * math.pi)
    if name == "gelu_tanh":
        p = _tanh_gate64(z)
        slope = 2.0 * math.sqrt(2.0 / math.pi) * (1.0 + 0.134145 * z * z)
        return p + z * p * (1.0 - p) * slope
    if name == "relu":
        return torch.where(z > 0, torch.ones_like(z), torch.zeros_like(z))
    return torch.ones_like(z)


def exact(case, seed):
    st = prepare(case, seed)
    d = {k: v.double() if isinstance(v, torch.Tensor) else v for k, v in st.items()}
    op = case["op"]
    if op in ("rotary", "heads", "heads_grad"):
        angle = torch.einsum("bs,i->bsi", d["positions"], d["inv_freq"]).unsqueeze(2)
        turn = torch.polar(torch.full_like(angle, st["scale"]), angle)
        out = {}
        for n in ("q", "k"):
            x = d[n]
            if op == "rotary":
                out[n] = _turned64(case, x, turn.conj() if case["inverse"] else turn)
                continue
            length = torch.sqrt(torch.einsum("bshd,bshd->bsh", x, x) / case["size"] + EPS)
            unit = x / length.unsqueeze(-1)
            gamma = d["gamma_" + n]
            if op == "heads":
                out[n] = _turned64(case, unit * gamma, turn)
                continue
            da = _turned64(case, d["d" + n], turn.conj())
            out["dgamma_" + n] = torch.einsum("bshd,bshd->d", da, unit)
            da = da * gamma
            along = torch.einsum("bshd,bshd->bsh", da, unit).unsqueeze(-1) / case["size"]
            out["d" + n] = (da - along * unit) / length.unsqueeze(-1)
        return out
    n, act = case["out"], case["act"]
    if op == "gated":
        z = torch.einsum("ri,oi->ro", d["x"], d["w"])
        if d["bias"] is not None:
            z = z + d["bias"]
        out = {"h": _value64(z[:, :n], act) * z[:, n:]}
        if case["keep"]:
            out["z"] = z
        return out
    gate, up = d["z"].split(n, 1)
    dz = torch.cat((d["dh"] * _derivative64(gate, act) * up, _value64(gate, act) * d["dh"]), 1)
    out = {"dx": torch.einsum("ro,oi->ri", dz, d["w"]), "dw": torch.einsum("ro,ri->oi", dz, d["x"])}
    if case["bias"]:
        out["db"] = dz.sum(dim=0)
    return out

"""What is measured of the layer-normalization and linear operators.

Four operators that together make a pre-norm MLP block on a residual stream, in
training and in serving:

  layer        S = x (+ skip (+ bias)); y = (S - mean) / sqrt(var + eps) * gamma + beta
  layer_grad   its gradients: of S, of gamma and beta, of bias
  linear       y = act(x W^T + b) + residual, with z = x W^T + b kept for training
  linear_grad  its gradients: of x, of W, of b

`own` chooses between the framework's kernels and the plain form in torch
operations.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
EPS = 1e-5
ACTIVATIONS = {"none": 0, "silu": 1, "gelu": 2, "gelu_tanh": 3, "relu": 4}

# Work of the largest listed case: linear_grad over a batch of 8 x 2048 tokens.
LARGEST_MACS = 2 * 16384 * 4096 * 16384


def _layer(name, rows, hidden, t, m, skip, bias, want_sum, stats):
    return {"name": name, "op": "layer", "rows": rows, "hidden": hidden, "t": t, "m": m,
            "skip": skip, "bias": bias, "sum": want_sum, "stats": stats}


def _layer_grad(name, rows, hidden, t, m, ds, dbias):
    return {"name": name, "op": "layer_grad", "rows": rows, "hidden": hidden, "t": t, "m": m,
            "ds": ds, "dbias": dbias}


def _linear(name, rows, n_in, n_out, t, act, bias, residual, keep):
    return {"name": name, "op": "linear", "rows": rows, "in": n_in, "out": n_out, "t": t,
            "act": act, "bias": bias, "residual": residual, "keep": keep}


def _linear_grad(name, rows, n_in, n_out, t, act):
    return {"name": name, "op": "linear_grad", "rows": rows, "in": n_in, "out": n_out, "t": t,
            "act": act}


def listed():
    return [
        # serving: one new token's residual add and norm between two products
        _layer("layer_decode_bf16_1x4096", 1, 4096, "bf16", "bf16", True, True, True, False),
        # a final norm without a residual add, at sizes that fit no vector; float32 weights
        _layer("layer_odd_bf16_3001x1027", 3001, 1027, "bf16", "f32", False, False, False, True),
        # training or prefill over 8 x 2048 tokens of the residual stream
        _layer("layer_fp16_16384x4096", 16384, 4096, "f16", "f16", True, True, True, True),
        # a small float32 model's training step
        _layer_grad("layer_grad_fp32_64x768", 64, 768, "f32", "f32", True, False),
        # ragged rows of an odd width, float16 with float32 weights
        _layer_grad("layer_grad_odd_fp16_1999x1027", 1999, 1027, "f16", "f32", False, False),
        # training over 8 x 2048 tokens: the stream's own gradient joins in, bias trained too
        _layer_grad("layer_grad_bf16_16384x4096", 16384, 4096, "bf16", "bf16", True, True),
        # serving: one token through the product that widens the stream
        _linear("linear_decode_bf16_1x4096x16384", 1, 4096, 16384, "bf16", "silu", True, False,
                False),
        # serving a batch of 64 tokens: the product back onto the stream
        _linear("linear_decode_fp16_64x4096x4096", 64, 4096, 4096, "f16", "none", True, True,
                False),
        # sizes that fit neither a tile nor a 16-byte row
        _linear("linear_odd_bf16_777x1027x1283", 777, 1027, 1283, "bf16", "gelu_tanh", True, True,
                True),
        # training or prefill over 8 x 2048 tokens
        _linear("linear_bf16_16384x4096x16384", 16384, 4096, 16384, "bf16", "gelu", True, False,
                True),
        # a small float32 model's training step (8 sequences of 64)
        _linear_grad("linear_grad_fp32_512x768x768", 512, 768, 768, "f32", "silu"),
        # training over 8 x 2048 tokens (the largest case)
        _linear_grad("linear_grad_bf16_16384x4096x16384", 16384, 4096, 16384, "bf16", "gelu"),
    ]


def _spread(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]; two in three are multiples of 64."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    if v >= 64 and rng.random() < 2 / 3:
        return min(hi, max(64, int(v) // 64 * 64))
    return min(hi, max(lo, int(v)))


def draw(rng):
    op = rng.choice(["layer", "layer_grad", "linear", "linear_grad"])
    t = rng.choice(["bf16", "f16", "f32"])
    if op in ("layer", "layer_grad"):
        rows, hidden = _spread(rng, 1, 16384), _spread(rng, 64, 16384)
        while rows * hidden > 16384 * 4096:
            rows, hidden = _spread(rng, 1, 16384), _spread(rng, 64, 16384)
        m = rng.choice([t, "f32"])
        if op == "layer":
            skip = rng.random() < 0.7
            c = _layer("", rows, hidden, t, m, skip, skip and rng.random() < 0.5,
                       skip and rng.random() < 0.7, rng.random() < 0.5)
        else:
            c = _layer_grad("", rows, hidden, t, m, rng.random() < 0.5, rng.random() < 0.5)
    else:
        most = LARGEST_MACS // (32 if t == "f32" else 4)
        while True:
            rows = _spread(rng, 1, 16384)
            n_in, n_out = _spread(rng, 64, 16384), _spread(rng, 64, 16384)
            if rows * n_in * n_out <= most:
                break
        act = rng.choice(sorted(ACTIVATIONS))
        if op == "linear":
            keep = rng.random() < 0.5
            c = _linear("", rows, n_in, n_out, t, act, rng.random() < 0.7, rng.random() < 0.5,
                        keep)
        else:
            c = _linear_grad("", rows, n_in, n_out, t, act)
    del c["name"]
    return c


class _Maker:
    """Random tensors from one seed, on the GPU."""

    def __init__(self, seed):
        self.gen = torch.Generator(device="cuda")
        self.gen.manual_seed(seed)

    def normal(self, shape, t, scale=1.0, mean=0.0):
        v = torch.randn(shape, generator=self.gen, device="cuda", dtype=torch.float32)
        return v.mul_(scale).add_(mean).to(DTYPES[t])


def _stream(mk, rows, hidden, t):
    """Rows of a residual stream: unit spread, an offset of their own, a few wide channels."""
    wide = torch.ones(hidden, device="cuda")
    wide[torch.randint(0, hidden, (max(1, hidden // 256),), generator=mk.gen, device="cuda")] = 8.0
    v = torch.randn((rows, hidden), generator=mk.gen, device="cuda", dtype=torch.float32)
    off = torch.randn((rows, 1), generator=mk.gen, device="cuda", dtype=torch.float32)
    return v.mul_(wide).add_(off.mul_(0.5)).to(DTYPES[t])


def prepare(case, seed):
    mk = _Maker(seed)
    st = {"case": case}
    op, t = case["op"], case["t"]
    if op in ("layer", "layer_grad"):
        rows, hidden, m = case["rows"], case["hidden"], case["m"]
        st["x"] = _stream(mk, rows, hidden, t)
        st["gamma"] = mk.normal((hidden,), m, 0.1, 1.0)
        if op == "layer":
            st["beta"] = mk.normal((hidden,), m, 0.1)
            st["skip"] = mk.normal((rows, hidden), t) if case["skip"] else None
            st["bias"] = mk.normal((hidden,), t, 0.1) if case["bias"] else None
        else:
            s = st["x"].double()
            st["mean"] = s.mean(1, keepdim=True)
            st["inv"] = (s.sub_(st["mean"]).square_().mean(1, keepdim=True) + EPS).rsqrt().float()
            st["mean"] = st["mean"].float()
            st["dy"] = mk.normal((rows, hidden), t, 0.1)
            st["ds"] = mk.normal((rows, hidden), t, 0.1) if case["ds"] else None
    else:
        rows, n_in, n_out = case["rows"], case["in"], case["out"]
        st["x"] = mk.normal((rows, n_in), t)
        st["w"] = mk.normal((n_out, n_in), t, 1.0 / math.sqrt(n_in))
        if op == "linear":
            st["bias"] = mk.normal((n_out,), t, 0.1) if case["bias"] else None
            st["residual"] = mk.normal((rows, n_out), t) if case["residual"] else None
        else:
            st["dy"] = mk.normal((rows, n_out), t, 0.1)
            st["z"] = mk.normal((rows, n_out), t) if case["act"] != "none" else None
    return st


# -- the plain form: binary32, one rounding at the end ------------------------

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
    if op == "layer":
        s = st["x"].float()
        if st["skip"] is not None:
            s = s + st["skip"].float()
            if st["bias"] is not None:
                s = s + st["bias"].float()
        stored = s.to(t)
        s = stored.float()
        mean = s.mean(1, keepdim=True)
        c = s - mean
        inv = torch.rsqrt((c * c).mean(1, keepdim=True) + EPS)
        y = (c * inv * st["gamma"].float() + st["beta"].float()).to(t)
        out = {"y": y}
        if case["sum"]:
            out["s"] = stored
        if case["stats"]:
            out["mean"], out["inv_std"] = mean, inv
        return out
    if op == "layer_grad":
        dy, gamma = st["dy"].float(), st["gamma"].float()
        xh = (st["x"].float() - st["mean"]) * st["inv"]
        g = dy * gamma
        dx = st["inv"] * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
        if st["ds"] is not None:
            dx = dx + st["ds"].float()
        m = DTYPES[case["m"]]
        out = {"dx": dx.to(t), "dgamma": (dy * xh).sum(0).to(m), "dbeta": dy.sum(0).to(m)}
        if case["dbias"]:
            out["dbias"] = dx.sum(0).to(t)
        return out
    x, w = st["x"].float(), st["w"].float()
    if op == "linear":
        z = x @ w.t()
        if st["bias"] is not None:
            z = z + st["bias"].float()
        y = _act(z, case["act"])
        if st["residual"] is not None:
            y = y + st["residual"].float()
        return {"y": y.to(t), "z": z.to(t)} if case["keep"] else {"y": y.to(t)}
    dz = st["dy"].float()
    if st["z"] is not None:
        dz = dz * _act_slope(st["z"].float(), case["act"])
    return {"dx": (dz @ w).to(t), "dw": (dz.t() @ x).to(t), "db": dz.sum(0).to(t)}


# -- the framework's kernels --------------------------------------------------

def _own(st):
    import residual_add_normalization_gb300 as b2
    case = st["case"]
    op = case["op"]
    if op == "layer":
        if case["stats"]:
            y, s, mean, inv = b2.skip_layer_stats(st["x"], st["skip"], st["gamma"], st["beta"],
                                                  st["bias"], epsilon=EPS, want_sum=case["sum"])
        else:
            y, s = b2.skip_layer(st["x"], st["skip"], st["gamma"], st["beta"], st["bias"],
                                 epsilon=EPS, want_sum=case["sum"])
        out = {"y": y}
        if case["sum"]:
            out["s"] = s
        if case["stats"]:
            out["mean"], out["inv_std"] = mean, inv
        return out
    if op == "layer_grad":
        dx, dgamma, dbeta, dbias = b2.skip_layer_grad(st["dy"], st["x"], st["mean"], st["inv"],
                                                      st["gamma"], ds=st["ds"],
                                                      want_bias=case["dbias"])
        out = {"dx": dx, "dgamma": dgamma, "dbeta": dbeta}
        if case["dbias"]:
            out["dbias"] = dbias
        return out
    act = ACTIVATIONS[case["act"]]
    if op == "linear":
        y, z = b2.linear(st["x"], st["w"], st["bias"], st["residual"], activation=act,
                         want_z=case["keep"])
        return {"y": y, "z": z} if case["keep"] else {"y": y}
    dx, dw, db = b2.linear_grad(st["dy"], st["x"], st["w"], st["z"], activation=act)
    return {"dx": dx, "dw": dw, "db": db}


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    es = SIZE[case["t"]]
    if case["op"] in ("layer", "layer_grad"):
        rows, hidden, ms = case["rows"], case["hidden"], SIZE[case["m"]]
        if case["op"] == "layer":
            tensors = 2 + case["skip"] + case["sum"]
            extra = hidden * (2 * ms + case["bias"] * es) + case["stats"] * 8 * rows
            flops = 8 * rows * hidden
        else:
            tensors = 3 + case["ds"]
            extra = hidden * (3 * ms + case["dbias"] * es) + 8 * rows
            flops = 14 * rows * hidden
        return {"bytes": rows * hidden * es * tensors + extra, "flops": flops}
    rows, n_in, n_out = case["rows"], case["in"], case["out"]
    if case["op"] == "linear":
        n = (rows * n_in + n_in * n_out + case["bias"] * n_out
             + rows * n_out * (1 + case["residual"] + case["keep"]))
        return {"bytes": n * es, "flops": 2 * rows * n_in * n_out}
    n = 2 * (rows * n_in + n_in * n_out) + n_out + rows * n_out * (1 + (case["act"] != "none"))
    return {"bytes": n * es, "flops": 4 * rows * n_in * n_out}


# -- the definitions in 64 bits -----------------------------------------------

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
    return torch.where(z > 0, torch.ones_like(z), torch.zeros_like(z))


def exact(case, seed):
    st = prepare(case, seed)
    d = {k: v.double() if isinstance(v, torch.Tensor) else v for k, v in st.items()}
    op = case["op"]
    if op == "layer":
        # S's own roundings are part of the definition: binary32 sums, one rounding to T
        total = st["x"].float()
        for name in ("skip", "bias"):
            if st[name] is not None:
                total = torch.add(total, st[name].float())
        kept = total.to(st["x"].dtype)
        s = kept.double()
        n = case["hidden"]
        mean = s.sum(dim=1, keepdim=True) / n
        var = ((s - mean) ** 2).sum(dim=1, keepdim=True) / n
        inv = 1.0 / torch.sqrt(var + EPS)
        out = {"y": (s - mean) * inv * d["gamma"] + d["beta"]}
        if case["sum"]:
            out["s"] = s
        if case["stats"]:
            out["mean"], out["inv_std"] = mean, inv
        return out
    if op == "layer_grad":
        n = case["hidden"]
        unit = (d["x"] - d["mean"]) * d["inv"]
        dunit = d["dy"] * d["gamma"]
        along = torch.einsum("rc,rc->r", dunit, unit).unsqueeze(1) / n
        dx = (dunit - dunit.sum(dim=1, keepdim=True) / n - along * unit) * d["inv"]
        if d["ds"] is not None:
            dx = dx + d["ds"]
        out = {"dx": dx, "dgamma": torch.einsum("rc,rc->c", d["dy"], unit),
               "dbeta": d["dy"].sum(dim=0)}
        if case["dbias"]:
            out["dbias"] = dx.sum(dim=0)
        return out
    if op == "linear":
        z = torch.einsum("ri,oi->ro", d["x"], d["w"])
        if d["bias"] is not None:
            z = z + d["bias"]
        y = _value64(z, case["act"])
        if d["residual"] is not None:
            y = y + d["residual"]
        return {"y": y, "z": z} if case["keep"] else {"y": y}
    dz = d["dy"] if d["z"] is None else d["dy"] * _derivative64(d["z"], case["act"])
    return {"dx": torch.einsum("ro,oi->ri", dz, d["w"]),
            "dw": torch.einsum("ro,ri->oi", dz, d["x"]), "db": dz.sum(dim=0)}

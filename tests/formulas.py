"""The layer-normalization and linear operators in binary64, from their
definitions, with bounds on how far a binary32 evaluation may be off.

Bounds count rounding steps: a stored value is off by at most half a step of
its type (HALF[t], relative; plus half the smallest subnormal), and a binary32
sum of n terms by at most (n - 1) half steps of the sum of the magnitudes,
whatever the order.  U is binary32's half step.
"""
import math

import torch

U = 2.0 ** -24
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ACTIVATIONS = {"none": 0, "silu": 1, "gelu": 2, "gelu_tanh": 3, "relu": 4}


def half(t):
    return torch.finfo(t).eps / 2


def stored(v, t):
    """How far rounding v to t may take it."""
    return v.abs() * half(t) + torch.finfo(t).smallest_normal * torch.finfo(t).eps / 2


# -- layer normalization ------------------------------------------------------

def residual_sum(x, skip, bias):
    """S: binary32 sums in order, one rounding to x's type."""
    if skip is None:
        return x
    s = x.float() + skip.float()
    if bias is not None:
        s = s + bias.float()
    return s.to(x.dtype)


def layer(s, gamma, beta, eps):
    """(y, mean, inv_std, bound on y's error before its rounding) in binary64."""
    s, gamma = s.double(), gamma.double()
    mean = s.mean(-1, keepdim=True)
    c = s - mean
    inv = 1.0 / torch.sqrt((c * c).mean(-1, keepdim=True) + eps)
    y = c * inv * gamma
    if beta is not None:
        y = y + beta.double()
    n = s.shape[-1]
    # longest chain of additions: the walk's per-thread run (at most one
    # vector of 8 per 512 threads and step) and its 10 butterfly steps
    depth = 8 * math.ceil(n / 4096) + n % 8 + 16
    dmean = depth * U * s.abs().mean(-1, keepdim=True)
    # the centred squares' mean shifts by dmean^2 and loses depth half steps
    dc = dmean + U * (s.abs() + mean.abs())
    bound = gamma.abs() * (inv * dc + (c * inv).abs() * (depth + 6) * U
                           + (c * inv).abs() * (inv * dmean) ** 2) + 4 * U * y.abs()
    if beta is not None:
        bound = bound + 2 * U * beta.double().abs()
    return y, mean, inv, bound


def layer_grad(dy, s, mean, inv, gamma, ds):
    """(dx, dgamma, dbeta, dbias) and the bounds on their errors before rounding."""
    dy, s, mean, inv, gamma = (v.double() for v in (dy, s, mean, inv, gamma))
    n, rows = s.shape[-1], s.shape[0]
    u = (s - mean) * inv
    g = dy * gamma
    c1 = g.sum(-1, keepdim=True) / n
    c2 = (g * u).sum(-1, keepdim=True) / n
    dx = inv * (g - c1 - u * c2)
    depth = 8 * math.ceil(n / 4096) + n % 8 + 20
    e1 = depth * U * g.abs().mean(-1, keepdim=True)
    e2 = depth * U * (g * u).abs().mean(-1, keepdim=True)
    bound = inv * (8 * U * (g.abs() + c1.abs() + (u * c2).abs()) + e1 + u.abs() * e2)
    if ds is not None:
        dx = dx + ds.double()
        bound = bound + U * dx.abs()
    steps = (rows + 20) * U
    return ((dx, (dy * u).sum(0), dy.sum(0), dx.sum(0)),
            (bound, steps * (dy * u).abs().sum(0), steps * dy.abs().sum(0),
             bound.sum(0) + steps * dx.abs().sum(0)))


# -- linear -------------------------------------------------------------------

def act(z, name):
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu":
        return z * 0.5 * torch.special.erfc(-z / math.sqrt(2.0))
    if name == "gelu_tanh":
        return z * 0.5 * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if name == "relu":
        return torch.clamp(z, min=0.0)
    return z


def act_grad(z, name):
    if name == "silu":
        s = torch.sigmoid(z)
        return s * (1 + z * (1 - s))
    if name == "gelu":
        return (0.5 * torch.special.erfc(-z / math.sqrt(2.0))
                + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi))
    if name == "gelu_tanh":
        k = math.sqrt(2 / math.pi)
        th = torch.tanh(k * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + th) + 0.5 * z * (1 - th * th) * k * (1 + 3 * 0.044715 * z * z)
    if name == "relu":
        return (z > 0).to(z.dtype)
    return torch.ones_like(z)


def linear(x, w, bias, residual, name):
    """(y, z) and the bounds on their errors before rounding."""
    x, w = x.double(), w.double()
    z = x @ w.t()
    mag = x.abs() @ w.abs().t()
    if bias is not None:
        z = z + bias.double()
        mag = mag + bias.double().abs()
    ez = (x.shape[-1] + 8) * U * mag
    y = act(z, name)
    # slopes stay below 1.13; the exponential's argument is off by half steps
    # of |z|, its value by a few more
    ey = 1.13 * ez + (z.abs() + 8) * 4 * U * y.abs()
    if residual is not None:
        ey = ey + 2 * U * (y.abs() + residual.double().abs())
        y = y + residual.double()
    return (y, z), (ey, ez)


def linear_grad(dy, x, w, z, name):
    """(dx, dw, db) and the bounds on their errors before rounding, for the
    unrounded dz: with an activation dz is rounded to its type on the way."""
    t = x.dtype
    dy, x, w = dy.double(), x.double(), w.double()
    dz, e = dy, torch.zeros_like(dy)
    if name != "none":
        zd = z.double()
        dz = dy * act_grad(zd, name)
        e = dy.abs() * (zd.abs() + 8) * 8 * U
    ez = e + (stored(dz, t) if name != "none" else 0)
    rows, out = dz.shape
    return ((dz @ w, dz.t() @ x, dz.sum(0)),
            (ez @ w.abs() + (out + 8) * U * ((dz.abs() + ez) @ w.abs()),
             ez.t() @ x.abs() + (rows + 8) * U * ((dz.abs() + ez).t() @ x.abs()),
             e.sum(0) + (rows + 20) * U * dz.abs().sum(0)))


# -- comparison ---------------------------------------------------------------

def assert_within(got, ref, bound, what):
    """Every element within `bound` plus its rounding; NaN meets NaN and
    infinities meet themselves."""
    t = got.dtype
    got = got.detach().cpu().double()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    tol = bound + stored(ref.abs() + bound, t)
    same = (got == ref) | (torch.isnan(got) & torch.isnan(ref))
    bad = ~(same | ((got - ref).abs() <= tol))
    if bad.any():
        i = tuple(int(k) for k in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {i}: "
                             f"got {got[i].item()!r}, want {ref[i].item()!r} +- {tol[i].item()!r}")


def assert_rms(got, ref, t, terms, what):
    """The error of the whole: rounding errors are spread evenly over a step, so
    their root mean square is half a step over sqrt(3) at most; `terms` is the
    number of binary32 additions behind an element, whose errors add as a
    random walk (4 steps of slack each)."""
    got = got.detach().cpu().double()
    off = (got - ref).norm() / ref.norm().clamp_min(1e-300)
    lim = 1.5 * half(t) + 4 * U * math.sqrt(terms + 16)
    assert off <= lim, f"{what}: relative error {off:.3g} over {lim:.3g}"

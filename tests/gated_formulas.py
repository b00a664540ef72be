"""The gated linear operator in binary64, with bounds on how far a binary32 evaluation may
be off before its rounding (formulas.py's counts: sums of n terms, activations off by a few
half steps of their argument)."""
import math

import torch

import formulas
from formulas import U, stored


# The tanh form of GELU by the logistic function, (1 + tanh w) / 2 = s(2 w): the sum 1 + tanh w
# keeps no digits of a gate's far tail in binary64 either.

def _two_w(z):
    return 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)


def act(z, name):
    return z * torch.sigmoid(_two_w(z)) if name == "gelu_tanh" else formulas.act(z, name)


def act_grad(z, name):
    if name != "gelu_tanh":
        return formulas.act_grad(z, name)
    p, q = torch.sigmoid(_two_w(z)), torch.sigmoid(-_two_w(z))
    return p + z * p * q * 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z * z)


def gated(x, w, bias, name):
    """(h, z) and the bounds on their errors before rounding."""
    x, w = x.double(), w.double()
    z = x @ w.t()
    mag = x.abs() @ w.abs().t()
    if bias is not None:
        z = z + bias.double()
        mag = mag + bias.double().abs()
    ez = (x.shape[-1] + 8) * U * mag
    n = z.shape[-1] // 2
    gate, up = z[:, :n], z[:, n:]
    a = act(gate, name)
    ea = 1.13 * ez[:, :n] + (gate.abs() + 8) * 4 * U * a.abs()
    h = a * up
    return (h, z), (ea * (up.abs() + ez[:, n:]) + a.abs() * ez[:, n:] + U * h.abs(), ez)


def dz_of(dh, z, name):
    """dz and the bound on its error before rounding."""
    dh, z = dh.double(), z.double()
    n = z.shape[-1] // 2
    gate, up = z[:, :n], z[:, n:]
    dz = torch.cat((dh * up * act_grad(gate, name), dh * act(gate, name)), -1)
    slope = (gate.abs() + 8) * 8 * U
    e = torch.cat(((dh * up).abs() * slope, (dh * act(gate, name)).abs() * slope), -1)
    # an exponential below binary32's smallest normal number, 2^-126, counts as zero (the
    # gate's tail): act and act' are then off by at most 2^-126 times z, or times z^2 and 1
    tiny = 2.0 ** -126 * (gate * gate + gate.abs() + 1)
    e = e + torch.cat(((dh * up).abs() * tiny, dh.abs() * tiny), -1)
    return dz, e + 2 * U * dz.abs()


def gated_grad(dh, x, w, z, name):
    """(dx, dw, db) and the bounds on their errors before rounding: dz is rounded to its type
    on the way to the products (bounds of more than four rows allow for that)."""
    t = x.dtype
    x, w = x.double(), w.double()
    dz, e = dz_of(dh, z, name)
    rows, out = dz.shape
    ez = e + stored(dz, t) if rows > 4 else e
    return ((dz @ w, dz.t() @ x, dz.sum(0)),
            (ez @ w.abs() + (out + 8) * U * ((dz.abs() + ez) @ w.abs()),
             ez.t() @ x.abs() + (rows + 8) * U * ((dz.abs() + ez).t() @ x.abs()),
             e.sum(0) + (rows + 20) * U * dz.abs().sum(0)))

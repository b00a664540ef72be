"""Rotation and RMS norm of heads in binary64, with bounds on how far a binary32
evaluation may be off before its rounding (U: binary32's half step).

Cosine and sine: the angle is reduced to an eighth of a turn exactly, up to 2^-32
turns; it is then off by 3 half steps of at most pi / 4, the series by 2.5e-8 and a
few half steps of its terms: 8 U in all, 9 U with the scale.  A rotated element is
two products and a sum: (|a| + |b|) * 12 U.  The inverse length: a sum of squares
(no cancellation; 32 terms in a lane at most, 5 butterfly steps, the mean: 40 half
steps), half of that in the root, whose own error is 2 last places: 24 U.
"""
import torch

from formulas import U

ROT, NORM = 12 * U, 27 * U


def turn_of(positions, inv_freq, scale):
    """exp(i p f) * scale, (..., 1, pairs), binary64."""
    angle = positions.double().unsqueeze(-1) * inv_freq.double()
    return torch.polar(torch.full_like(angle, scale), angle).unsqueeze(-2)


def rotate(v, turn, interleaved):
    """(rotated v, |a| + |b| of each element's pair, 0 past the pairs)."""
    h = turn.shape[-1]
    out, mag = v.clone(), torch.zeros_like(v)
    if h == 0:
        return out, mag
    one, two = ((slice(0, 2 * h, 2), slice(1, 2 * h, 2)) if interleaved
                else (slice(0, h), slice(h, 2 * h)))
    a, b = v[..., one], v[..., two]
    c, s = turn.real, turn.imag
    out[..., one], out[..., two] = a * c - b * s, b * c + a * s
    m = (a.abs() + b.abs()) * turn.abs()
    mag[..., one] = m
    mag[..., two] = m
    return out, mag


def rotary(x, turn, interleaved):
    y, mag = rotate(x.double(), turn, interleaved)
    return y, mag * ROT


def head_norm(x, gamma, turn, eps, interleaved):
    x = x.double()
    a = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    if gamma is not None:
        a = a * gamma.double()
    y, mag = rotate(a, turn, interleaved)
    plain = torch.where(mag == 0, a.abs(), torch.zeros_like(a)) * NORM
    return y, mag * (ROT + NORM) + plain


def head_norm_grad(dy, x, gamma, turn, eps, interleaved):
    """(dx, dgamma) and the bounds on their errors."""
    dy, x = dy.double(), x.double()
    g = torch.ones(x.shape[-1], dtype=torch.float64) if gamma is None else gamma.double()
    r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    u = x * r
    da, mag = rotate(dy, turn.conj(), interleaved)
    ea = mag * ROT
    gu = da * g
    eg = ea * g.abs() + U * gu.abs()
    m = (gu * u).mean(-1, keepdim=True)
    em = ((gu * u).abs().mean(-1, keepdim=True) * (NORM + 40 * U)
          + (eg * u.abs()).mean(-1, keepdim=True))
    dx = r * (gu - m * u)
    ex = (r * (eg + (m * u).abs() * NORM + em * u.abs() + 3 * U * (gu.abs() + (m * u).abs()))
          + NORM * dx.abs())
    rows = x[..., 0].numel()
    flat = lambda v: v.reshape(-1, v.shape[-1]).sum(0)  # noqa: E731
    dgamma = flat(da * u)
    eg = (rows + 40) * U * flat((da * u).abs()) + flat(ea * u.abs() + (da * u).abs() * NORM)
    return (dx, dgamma), (ex, eg)

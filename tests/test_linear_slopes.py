"""The derivatives of the linear operator's activations, an element at a time: db
of a single row with dy = 1 is act'(z) itself.

Bounds count half steps of binary32 (U).  The hardware's exponential is off by 4 U
relative (2^-22), its reciprocal by 2 U (2^-23); a relative error ea of the
exponential's argument a costs |a| * ea, and the product with log2(e) 2 U more.
With e = exp(-|a|), p = s(a), q = 1 - p:

  e    (ea + 2) |a| + 4 =: E
  p    the larger of p and q is 1 / (1 + e): its share of E is pq, and 3 for the
       sum and the reciprocal; the smaller, at most 2 pq, has E of its own and a
       product: in all 3 pq E + 4 p
  pq   2 E and 3 + 3 + 1

SiLU (a = z, exact): d = p + z p q, two products more: |z p q| (2 E + 9).
GELU tanh (a = K (z + C z^3): five products and sums and two constants, ea = 7):
d = p + z p q K (1 + 3 C z^2), at most twelve more: |second term| (2 E + 19).
GELU: d = P(z) + z f(z).  f's exponent has two products and a constant, 1.5 z^2,
and the exponential's 4; P's tail has that, the fit's 3, the reciprocal's 2, and
at most 20 from eight products and sums whose terms add up to less than twice the
value.
Each d is rounded once more, |d|; values too small for the hardware's normal range
are left out by an absolute 2^-100."""
import math

import pytest
import torch

import formulas as F
import residual_add_normalization_gb300 as b2

pytestmark = pytest.mark.gpu


def slope(z, name):
    """act'(z) in binary64 without cancellation, and its bound in half steps."""
    if name == "gelu":
        f = torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        tail = 0.5 * torch.special.erfc(z.abs() / math.sqrt(2.0))
        p = torch.where(z >= 0, 1 - tail, tail)
        d = p + z * f
        return d, tail * (1.5 * z * z + 32) + (z * f).abs() * (1.5 * z * z + 7) + p + d.abs()
    k, c = 2 * math.sqrt(2 / math.pi), 0.044715
    a = z if name == "silu" else k * (z + c * z ** 3)
    e = torch.exp(-a.abs())
    big, small = 1 / (1 + e), e / (1 + e)
    p, q = torch.where(a >= 0, big, small), torch.where(a >= 0, small, big)
    if name == "silu":
        second, off, more = z * p * q, 2 * a.abs() + 4, 9
    else:
        second, off, more = z * p * q * k * (1 + 3 * c * z * z), 9 * a.abs() + 4, 19
    d = p + second
    return d, 3 * p * q * off + 4 * p + second.abs() * (2 * off + more) + d.abs()


@pytest.mark.parametrize("name", ["silu", "gelu", "gelu_tanh"])
def test_slope(name):
    g = torch.Generator().manual_seed(1)
    far = torch.empty(100_000).uniform_(-103.9, 103.9, generator=g) if name == "silu" else \
        torch.empty(100_000).uniform_(-15.99, 15.99, generator=g)
    z = torch.cat([torch.linspace(-15.99, 15.99, 300_001), far,
                   torch.empty(100_000).uniform_(3, 16, generator=g),
                   torch.randn(20_000, generator=g) * 1e-3, torch.zeros(1)]).float()
    n = z.numel()
    one = torch.ones(n, device="cuda")
    _, _, db = b2.linear_grad(one.view(1, n), one[:1].view(1, 1), one.view(n, 1),
                              z.cuda().view(1, n), activation=F.ACTIVATIONS[name],
                              want_input=False, want_weight=False)
    want, steps = slope(z.double(), name)
    off = (db.cpu().double() - want).abs()
    tol = 1.01 * F.U * steps + 2.0 ** -100
    worst = int((off / tol).argmax())
    assert bool((off <= tol).all()), (z[worst].item(), off[worst].item() / F.U,
                                      tol[worst].item() / F.U)

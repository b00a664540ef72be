"""GPU: the column sums of the gradient of layer normalization, exactly.

With whole numbers in dy, s and ds, a mean of 0, an inv_std_var of 1 and a gamma of
0, u = s and dx = ds, and dgamma, dbeta and dbias are sums of whole numbers that
binary32 holds exactly in any order (|terms| <= 9, below 2^24 in all).  A row that
is left out, taken twice or taken from another place changes them."""
import pytest
import torch

import formulas as F
import residual_add_normalization_gb300 as b2
from test_layer import ODD_SHAPES, SHAPES, TYPES

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _no_wait_gave_up():
    yield
    b2.rows_status()


def whole(shape, t, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-3, 4, shape, generator=g, device="cuda", dtype=torch.int8).to(t)


def sums(rows, hidden, *terms):
    """Column sums of a product of tensors, in binary64, some rows at a time."""
    out = torch.zeros(hidden, dtype=torch.float64, device="cuda")
    step = max(1, (1 << 26) // hidden)
    for a in range(0, rows, step):
        p = terms[0][a:a + step].double()
        for t in terms[1:]:
            p = p * t[a:a + step].double()
        out += p.sum(0)
    return out


def check(rows, hidden, t, m, bias=True, shift=0):
    def at(v):  # starting `shift` elements into its block
        flat = torch.empty(v.numel() + shift, dtype=v.dtype, device="cuda")
        out = flat[shift:].view(v.shape)
        return out.copy_(v)
    dy, s, ds = (at(whole((rows, hidden), t, rows + hidden + i)) for i in range(3))
    mean, inv = torch.zeros(rows, 1, device="cuda"), torch.ones(rows, 1, device="cuda")
    gamma = torch.zeros(hidden, dtype=m, device="cuda")
    dx, dgamma, dbeta, dbias = b2.skip_layer_grad(dy, s, mean, inv, gamma, ds=ds, want_bias=bias)
    assert torch.equal(dx, ds)
    assert torch.equal(dgamma, sums(rows, hidden, dy, s).to(m))
    assert torch.equal(dbeta, sums(rows, hidden, dy).to(m))
    if bias:
        assert torch.equal(dbias, sums(rows, hidden, ds).to(t))


LONG = [(400, 9000), (300, 16384), (130, 32768), (50, 65536), (70, 70001)]
MANY = [(40001, 64), (30000, 128), (20401, 768), (16384, 1024), (5000, 4096), (3001, 1040)]


@pytest.mark.parametrize("t,m", TYPES)
@pytest.mark.parametrize("rows,hidden", SHAPES + ODD_SHAPES + LONG + MANY)
def test_exact(rows, hidden, t, m):
    check(rows, hidden, F.DTYPES[t], F.DTYPES[m])
    check(rows, hidden, F.DTYPES[t], F.DTYPES[m], bias=False)


@pytest.mark.parametrize("t,m", TYPES)
@pytest.mark.parametrize("rows,hidden", [(9, 64), (3000, 1024), (20400, 131), (700, 4095),
                                         (141, 20001)])
def test_exact_unaligned(rows, hidden, t, m):
    check(rows, hidden, F.DTYPES[t], F.DTYPES[m], shift=1)


@pytest.mark.parametrize("hidden", [4096, 4095])
def test_exact_past_2_31_elements(hidden):
    check((1 << 31) // hidden + 77, hidden, torch.bfloat16, torch.float32)


@pytest.mark.parametrize("t,m", TYPES)
@pytest.mark.parametrize("rows,hidden", [(40001, 67), (20400, 131), (16384, 768), (3000, 1027)])
def test_error_of_the_whole(rows, hidden, t, m):
    """Ordinary values: the sums' errors add up as a random walk."""
    g = torch.Generator(device="cuda").manual_seed(rows)
    dy, s, ds = (torch.randn(rows, hidden, generator=g, device="cuda").to(F.DTYPES[t])
                 for _ in range(3))
    gamma = torch.rand(hidden, generator=g, device="cuda").to(F.DTYPES[m]) + 0.5
    _, _, mean, inv = b2.skip_layer_stats(s, None, gamma)
    got = b2.skip_layer_grad(dy, s, mean, inv, gamma, ds=ds, want_bias=True)
    want, _ = F.layer_grad(dy, s, mean, inv, gamma, ds)
    for name, p, q in zip(("dx", "dgamma", "dbeta", "dbias"), got, want):
        F.assert_rms(p, q.cpu(), p.dtype, hidden if name == "dx" else rows, name)

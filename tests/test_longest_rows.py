"""Rows of 2^31 - 1 elements, the longest that the row operators take: a row that is
not whole 16-byte vectors is walked an element at a time, and the walk's counter
passes 2^31.  The values are small whole numbers, so that every partial sum of a
row is exact in binary32, and the last elements are large, so that a row cut short
shows in the statistics."""
import pytest
import torch

import formulas as F
import residual_add_normalization_gb300 as b2

pytestmark = pytest.mark.gpu

N = (1 << 31) - 1
CHUNK = 1 << 27


def digits(seed, lo=-1, hi=2):
    """One row of whole numbers in [lo, hi) as bfloat16."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    v = torch.empty(1, N, dtype=torch.bfloat16, device="cuda")
    for a in range(0, N, CHUNK):
        b = min(N, a + CHUNK)
        v[0, a:b] = torch.randint(lo, hi, (b - a,), generator=g, device="cuda", dtype=torch.int8)
    return v


def chunks(*rows):
    """The same stretch of each row, widened to binary64, one after another."""
    for a in range(0, N, CHUNK):
        yield [r.view(-1)[a:a + CHUNK].double() for r in rows]


@pytest.fixture(scope="module")
def row():
    if torch.cuda.mem_get_info()[0] < 120e9:
        pytest.skip("not enough device memory")
    x = digits(1)
    x[0, -2:] = torch.tensor([64.0, 128.0])
    yield x
    torch.cuda.empty_cache()


def check(got, want, slack):
    """Half a step of bfloat16, and `slack` relative for the binary32 arithmetic."""
    tol = want.abs() * (F.half(torch.bfloat16) + slack) + 2.0 ** -120
    assert bool(((got - want).abs() <= tol).all())


def test_layer(row):
    gamma = torch.full((N,), 1.5, dtype=torch.bfloat16, device="cuda")
    y, s, mean, inv = b2.skip_layer_stats(row, None, gamma)
    assert s is row
    total = sum(int(c.sum()) for c, in chunks(row))
    mu = total / N
    # exact sums, one product with 1 / n: two half steps, and one of 1 / n
    assert abs(mean.item() - mu) <= 4 * F.U * abs(mu)
    var = sum(float(((c - mu) ** 2).sum()) for c, in chunks(row)) / N
    # squares: four million positive terms per thread, whose partial sums stay below
    # 2^22 and whose roundings to nearest are as often up as down
    assert abs(inv.item() - (var + 1e-5) ** -0.5) <= 1e-3 * inv.item()
    m, r = float(mean), float(inv)
    for got, c in chunks(y, row):
        # a difference, two products; the difference may cancel down to mu
        check(got, (c - m) * r * 1.5, 6 * F.U)


def test_layer_grad(row):
    gamma = torch.ones(N, dtype=torch.bfloat16, device="cuda")
    dy = digits(2)
    dy[0, -1] = 32.0
    mean = torch.full((1, 1), 0.25, device="cuda")
    inv = torch.full((1, 1), 0.5, device="cuda")
    dx, dgamma, dbeta, _ = b2.skip_layer_grad(dy, row, mean, inv, gamma)
    c1 = sum(int(d.sum()) for d, in chunks(dy)) / N
    c2 = sum(float((d * (x - 0.25) * 0.5).sum()) for d, x in chunks(dy, row)) / N
    for got, d, x in chunks(dx, dy, row):
        u = (x - 0.25) * 0.5
        # the sum of g * u is of multiples of 1/8 below 2^21: exact; three products
        # and two sums of terms that may cancel
        want = 0.5 * (d - c1 - u * c2)
        slack = 8 * F.U * (d.abs() + abs(c1) + (u * c2).abs())
        tol = (want.abs() + slack) * F.half(torch.bfloat16) + slack + 2.0 ** -120
        assert bool(((got - want).abs() <= tol).all())
    for g, b, d, x in chunks(dgamma, dbeta, dy, row):
        assert torch.equal(b, d)
        check(g, d * (x - 0.25) * 0.5, 0.0)


def test_skip_rms(row):
    skip = digits(3)
    gamma = torch.full((N,), 1.5, dtype=torch.bfloat16, device="cuda")
    y, s, _, inv = b2.skip_rms_stats(row, skip, gamma, epsilon=1e-5)
    squares = 0
    for got, a, b in chunks(s, row, skip):
        assert torch.equal(got, a + b)
        squares += int(((a + b) ** 2).sum())
    # a thread's sum stays below 2^24 and is exact; ten sums of threads and warps, the
    # mean, epsilon, and the reciprocal square root (2 half steps) of half of these
    r = (squares / N + 1e-5) ** -0.5
    assert abs(inv.item() - r) <= 10 * F.U * r
    for got, c in chunks(y, s):
        check(got, c * inv.item() * 1.5, 3 * F.U)


def test_gated_rms(row):
    gate = digits(4)
    scale = torch.full((N,), 1.5, dtype=torch.bfloat16, device="cuda")
    y = b2.gated_rms(row, gate, scale, epsilon=1e-5)
    r = (sum(int((c ** 2).sum()) for c, in chunks(row)) / N + 1e-5) ** -0.5
    for got, c, z in chunks(y, row, gate):
        # r's 10 half steps; SiLU's exponential (2 |z| + 4), sum, reciprocal (2) and
        # product; three products more
        check(got, c * r * 1.5 * z * torch.sigmoid(z), 24 * F.U)

"""GPU: layer normalization and the linear operator at their limits: waits that
give up, more elements than 2^31, and equal bits from equal calls."""
import time

import pytest
import torch

import formulas as F
import residual_add_normalization_gb300 as b2

pytestmark = pytest.mark.gpu

TIMEOUT = 5
LIMIT_NS = 20_000_000


@pytest.fixture(autouse=True)
def _normal_launches():
    yield
    lib = b2.library()
    lib.b200norm_testing_linear_stall(0, 0)
    lib.b200norm_testing_pipe_stall(0, 0)
    lib.b200norm_testing_force_linear(0, 0, 0, 0)
    b2.linear_status()
    b2.rows_status()


@pytest.mark.parametrize("tiling", [(2, 256, 1, 0), (1, 128, 1, 0), (1, 128, 4, 0), (1, 64, 2, 0),
                                    (1, 16, 2, 1)])
def test_linear_waits_give_up(tiling):
    """With nothing copied, the roles' waits run out: the call returns, the status
    says so once, and the next call is right."""
    lib = b2.library()
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(16, 1024, generator=g, device="cuda").bfloat16()
    w = torch.randn(600, 1024, generator=g, device="cuda").bfloat16()
    assert lib.b200norm_testing_force_linear(*tiling) == 0
    want, _ = b2.linear(x, w)
    b2.linear_status()
    assert lib.b200norm_testing_linear_stall(1, LIMIT_NS) == 0
    t0 = time.monotonic()
    b2.linear(x, w)
    with pytest.raises(b2.B200NormError) as e:
        b2.linear_status()
    assert e.value.status == TIMEOUT
    assert time.monotonic() - t0 < 2.0
    b2.linear_status()  # read and cleared
    assert lib.b200norm_testing_linear_stall(0, 0) == 0
    got, _ = b2.linear(x, w)
    b2.linear_status()
    assert torch.equal(got, want)


@pytest.mark.parametrize("rows,hidden,t", [(300, 4096, torch.bfloat16), (300, 64, torch.float32),
                                           (20, 20000, torch.float16), (90, 1027, torch.float16)])
def test_layer_gradient_waits_give_up(rows, hidden, t):
    lib = b2.library()
    g = torch.Generator(device="cuda").manual_seed(2)
    x, dy = (torch.randn(rows, hidden, generator=g, device="cuda").to(t) for _ in range(2))
    gamma = torch.ones(hidden, device="cuda")
    _, s, mean, inv = b2.skip_layer_stats(x, None, gamma)
    want = b2.skip_layer_grad(dy, s, mean, inv, gamma)
    b2.rows_status()
    assert lib.b200norm_testing_pipe_stall(1, LIMIT_NS) == 0
    t0 = time.monotonic()
    b2.skip_layer_grad(dy, s, mean, inv, gamma)
    with pytest.raises(b2.B200NormError) as e:
        b2.rows_status()
    assert e.value.status == TIMEOUT
    assert time.monotonic() - t0 < 2.0
    assert lib.b200norm_testing_pipe_stall(0, 0) == 0
    got = b2.skip_layer_grad(dy, s, mean, inv, gamma)
    b2.rows_status()
    assert all(torch.equal(p, q) for p, q in zip(got[:3], want[:3]))


def test_layer_past_2_31_elements():
    """Offsets that need more than 32 bits: the last rows against the formulas,
    and against the same rows by themselves."""
    rows, hidden = (1 << 31) // 4096 + 77, 4096
    x = torch.empty(rows, hidden, dtype=torch.bfloat16, device="cuda").normal_()
    gamma, beta = (torch.rand(hidden, device="cuda").bfloat16() for _ in range(2))
    y, _, mean, inv = b2.skip_layer_stats(x, None, gamma, beta)
    n = 5
    ref, rmean, rinv, bound = F.layer(x[-n:].cpu(), gamma.cpu(), beta.cpu(), 1e-5)
    F.assert_within(y[-n:], ref, bound, "y")
    dx, dgamma, dbeta, _ = b2.skip_layer_grad(y, x, mean, inv, gamma)
    some, _, _, _ = b2.skip_layer_grad(y[-n:].contiguous(), x[-n:].contiguous(),
                                       mean[-n:].contiguous(), inv[-n:].contiguous(), gamma)
    assert torch.equal(dx[-n:], some)
    # column sums over half a million rows: binary64 on the GPU, a column block
    dy64 = y[:, :8].double()
    want = dy64.sum(0)
    mag = dy64.abs().sum(0)
    assert bool(((dbeta[:8].double() - want).abs()
                 <= (rows / 152 + 2000) * F.U * mag + 2.0 ** -8 * want.abs()).all())


def test_linear_past_2_31_elements():
    rows, n_in, n_out = (1 << 31) // 16384 + 77, 64, 16384
    x = torch.empty(rows, n_in, dtype=torch.bfloat16, device="cuda").normal_()
    w = torch.empty(n_out, n_in, dtype=torch.bfloat16, device="cuda").normal_() / 8
    bias = torch.empty(n_out, dtype=torch.bfloat16, device="cuda").normal_()
    y, z = b2.linear(x, w, bias, activation=4, want_z=True)
    n = 3
    (ry, rz), (ey, ez) = F.linear(x[-n:].cpu(), w.cpu(), bias.cpu(), None, "relu")
    F.assert_within(y[-n:], ry, ey, "y")
    F.assert_within(z[-n:], rz, ez, "z")
    dx, _, _ = b2.linear_grad(y, x, w, z, activation=4, want_weight=False, want_bias=False)
    (rdx, _, _), (edx, _, _) = F.linear_grad(y[-n:].cpu(), x[-n:].cpu(), w.cpu(), z[-n:].cpu(),
                                             "relu")
    F.assert_within(dx[-n:], rdx, edx, "dx")


@pytest.mark.parametrize("t", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,n_in,n_out", [(1, 512, 768), (130, 1024, 520)])
def test_same_results_without_dependent_launch(rows, n_in, n_out, t):
    g = torch.Generator(device="cuda").manual_seed(4)
    x, w, dy = (torch.randn(*s, generator=g, device="cuda").to(t)
                for s in ((rows, n_in), (n_out, n_in), (rows, n_out)))
    gamma = torch.rand(n_in, generator=g, device="cuda").to(t)

    def run():
        n, s, mean, inv = b2.skip_layer_stats(x, x, gamma)
        y, z = b2.linear(n, w, activation=2, want_z=True)
        dn, dw, db = b2.linear_grad(dy, n, w, z, activation=2)
        return (y, z, dn, dw, db) + b2.skip_layer_grad(dn, s, mean, inv, gamma, want_bias=True)
    first = run()
    try:
        assert b2.library().b200norm_testing_set_pdl(0) == 0
        second = run()
    finally:
        b2.library().b200norm_testing_set_pdl(1)
    assert all(torch.equal(p, q) for p, q in zip(first, second))


@pytest.mark.parametrize("t", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,n_in,n_out", [(2, 512, 768), (40, 4096, 512), (700, 1027, 520)])
def test_equal_calls_give_equal_bits(rows, n_in, n_out, t):
    g = torch.Generator(device="cuda").manual_seed(3)
    x, w, dy = (torch.randn(*s, generator=g, device="cuda").to(t)
                for s in ((rows, n_in), (n_out, n_in), (rows, n_out)))
    gamma = torch.rand(n_in, generator=g, device="cuda").to(t)

    def run():
        n, s, mean, inv = b2.skip_layer_stats(x, x, gamma)
        y, z = b2.linear(n, w, activation=3, want_z=True)
        dn, dw, db = b2.linear_grad(dy, n, w, z, activation=3)
        return (y, z, dn, dw, db) + b2.skip_layer_grad(dn, s, mean, inv, gamma, want_bias=True)
    first = run()
    for _ in range(5):
        assert all(torch.equal(p, q) for p, q in zip(first, run()))

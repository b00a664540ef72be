"""CPU: what the layer and linear entry points refuse, before any CUDA call, and
the binary64 formulas that the GPU tests use, against differences."""
import pytest
import torch

import formulas as F
import residual_add_normalization_gb300 as b2
from residual_add_normalization_gb300 import buildlib

OK, INVALID, UNSUPPORTED, CUDA, WORKSPACE, TIMEOUT = range(6)
F32, F16, BF16 = 0, 1, 2
G = 1 << 30
FAKE = 1 << 40  # never dereferenced: every call below fails validation or is empty


@pytest.fixture(scope="module")
def lib():
    buildlib.build()
    return b2.library()


def layer(lib, **kw):
    a = dict(x=FAKE, skip=FAKE + G, gamma=FAKE + 2 * G, beta=None, bias=None, y=FAKE + 3 * G,
             s=None, mean=None, inv=None, rows=4, hidden=64, T=F16, M=F16, eps=1e-5)
    a.update(kw)
    return lib.b200norm_skip_layer(*a.values(), None)


def test_skip_layer_refusals(lib):
    assert layer(lib, T=3, M=3) == UNSUPPORTED
    assert layer(lib, M=BF16) == UNSUPPORTED            # bfloat16 gamma under float16 rows
    assert layer(lib, T=F32, M=F16) == UNSUPPORTED
    assert layer(lib, rows=-1) == INVALID
    assert layer(lib, hidden=0) == INVALID
    assert layer(lib, hidden=1 << 31) == UNSUPPORTED
    assert layer(lib, rows=1 << 31) == UNSUPPORTED
    assert layer(lib, eps=-1.0) == INVALID
    assert layer(lib, eps=float("nan")) == INVALID
    assert layer(lib, x=None) == INVALID
    assert layer(lib, gamma=None) == INVALID
    assert layer(lib, y=None) == INVALID
    assert layer(lib, x=FAKE + 1) == INVALID
    assert layer(lib, M=F32, gamma=FAKE + 2 * G + 2) == INVALID
    assert layer(lib, mean=FAKE + 4 * G + 2) == INVALID
    assert layer(lib, y=FAKE + 64) == INVALID           # over the input
    assert layer(lib, s=FAKE + 3 * G) == INVALID        # over the other output
    assert layer(lib, mean=FAKE + 4 * G, inv=FAKE + 4 * G + 8) == INVALID
    assert layer(lib, skip=None, bias=FAKE + 5 * G) == INVALID
    assert layer(lib, skip=None, s=FAKE + 5 * G) == INVALID
    assert b"need a skip" in lib.b200norm_last_error()
    assert layer(lib, rows=0, x=None, skip=None, gamma=None, y=None) == OK


def layer_grad(lib, **kw):
    a = dict(dy=FAKE, s=FAKE + G, mean=FAKE + 2 * G, inv=FAKE + 2 * G + 4096,
             gamma=FAKE + 3 * G, ds=None, dx=FAKE + 4 * G, dgamma=FAKE + 5 * G,
             dbeta=FAKE + 6 * G, dbias=None, rows=4, hidden=64, T=F16, M=F32,
             ws=FAKE + 7 * G, wsb=1 << 20)
    a.update(kw)
    return lib.b200norm_skip_layer_grad(*a.values(), None)


def test_skip_layer_grad_refusals(lib):
    assert layer_grad(lib, T=7) == UNSUPPORTED
    assert layer_grad(lib, M=BF16) == UNSUPPORTED
    assert layer_grad(lib, rows=-1) == INVALID
    assert layer_grad(lib, hidden=0) == INVALID
    for k in ("dy", "s", "mean", "inv", "gamma"):
        assert layer_grad(lib, **{k: None}) == INVALID, k
    assert layer_grad(lib, dx=FAKE) == INVALID                 # over dy
    assert layer_grad(lib, dbeta=FAKE + 5 * G + 4) == INVALID  # over dgamma
    assert layer_grad(lib, dgamma=FAKE + 5 * G + 1) == INVALID
    assert layer_grad(lib, ws=None) == WORKSPACE
    assert layer_grad(lib, wsb=8) == WORKSPACE
    assert layer_grad(lib, ws=FAKE + 7 * G + 64) == WORKSPACE
    assert layer_grad(lib, ws=FAKE) == WORKSPACE               # over dy
    # nothing wanted: nothing to do
    assert layer_grad(lib, dx=None, dgamma=None, dbeta=None) == OK


def test_layer_grad_workspace_size(lib):
    f = lib.b200norm_skip_layer_grad_workspace_size
    assert f(-1, 64) == 0 and f(4, 0) == 0
    # the row coefficients and at least one set of column sums
    for rows in (1, 100, 16384):
        for hidden in (1, 768, 1 << 20):
            assert f(rows, hidden) >= rows * 8 + 3 * hidden * 4


def linear(lib, **kw):
    a = dict(x=FAKE, w=FAKE + G, bias=None, residual=None, y=FAKE + 2 * G, z=None, rows=4,
             n_in=64, n_out=32, T=BF16, act=0, ws=FAKE + 3 * G, wsb=1 << 24)
    a.update(kw)
    return lib.b200norm_linear(*a.values(), None)


def test_linear_refusals(lib):
    assert linear(lib, T=3) == UNSUPPORTED
    assert linear(lib, rows=-1) == INVALID
    assert linear(lib, n_in=0) == INVALID
    assert linear(lib, n_out=0) == INVALID
    assert linear(lib, n_out=(1 << 20) + 1) == UNSUPPORTED
    assert linear(lib, rows=1 << 31) == UNSUPPORTED
    assert linear(lib, rows=(1 << 30) + 1) == UNSUPPORTED
    assert linear(lib, act=5) == INVALID
    assert linear(lib, act=-1) == INVALID
    assert linear(lib, x=None) == INVALID
    assert linear(lib, w=None) == INVALID
    assert linear(lib, y=None) == INVALID
    assert linear(lib, w=FAKE + G + 1) == INVALID
    assert linear(lib, y=FAKE + 2) == INVALID                 # over x
    assert linear(lib, z=FAKE + 2 * G + 2) == INVALID         # over y
    assert linear(lib, residual=FAKE + 2 * G) == INVALID      # y may not be updated in place
    assert linear(lib, rows=0, x=None, w=None, y=None, ws=None, wsb=0) == OK


def linear_grad(lib, **kw):
    a = dict(dy=FAKE, x=FAKE + G, w=FAKE + 2 * G, z=FAKE + 3 * G, dx=FAKE + 4 * G,
             dw=FAKE + 5 * G, db=FAKE + 6 * G, rows=4, n_in=64, n_out=32, T=BF16, act=1,
             ws=FAKE + 7 * G, wsb=1 << 24)
    a.update(kw)
    return lib.b200norm_linear_grad(*a.values(), None)


def test_linear_grad_refusals(lib):
    assert linear_grad(lib, T=3) == UNSUPPORTED
    assert linear_grad(lib, rows=-1) == INVALID
    assert linear_grad(lib, act=9) == INVALID
    for k in ("dy", "x", "w", "z"):
        assert linear_grad(lib, **{k: None}) == INVALID, k
    assert linear_grad(lib, dw=FAKE + G) == INVALID           # over x
    assert linear_grad(lib, db=FAKE + 5 * G) == INVALID       # over dw
    assert linear_grad(lib, dx=FAKE + 4 * G + 1) == INVALID
    assert linear_grad(lib, ws=None) == WORKSPACE
    assert linear_grad(lib, wsb=16) == WORKSPACE
    assert linear_grad(lib, ws=FAKE + 7 * G + 16) == WORKSPACE
    assert linear_grad(lib, ws=FAKE + 2 * G) == WORKSPACE     # over weight
    assert linear_grad(lib, dx=None, dw=None, db=None) == OK


def test_linear_workspace_sizes(lib):
    assert lib.b200norm_linear_workspace_size(4, 0, 8, BF16, 1) == 0
    # with an activation, dz is kept
    with_act = lib.b200norm_linear_grad_workspace_size(64, 128, 256, BF16, 2, 1)
    assert with_act >= 64 * 256 * 2
    assert lib.b200norm_linear_grad_workspace_size(64, 128, 256, BF16, 9, 1) == 0


def test_force_hook_refusals(lib):
    f = lib.b200norm_testing_force_linear
    for bad in ((3, 64, 1, 0), (1, 48, 1, 0), (1, 64, 3, 0), (1, 64, 1, 2), (0, 64, 1, 0)):
        assert f(*bad) == INVALID, bad
    assert f(1, 64, 8, 0) == OK
    assert f(0, 0, 0, 0) == OK


def test_stall_hook_refusals(lib):
    f = lib.b200norm_testing_linear_stall
    assert f(2, 1000) == INVALID
    assert f(1, 0) == INVALID
    assert f(1, 6_000_000_000) == INVALID
    assert f(0, 0) == OK


def test_binding_refuses_cpu_tensors():
    x, w = torch.zeros(4, 8), torch.ones(8)
    with pytest.raises(ValueError, match="CUDA"):
        b2.skip_layer(x, x, w)
    with pytest.raises(ValueError, match="CUDA"):
        b2.skip_layer_grad(x, x, torch.zeros(4, 1), torch.ones(4, 1), w)
    with pytest.raises(ValueError, match="CUDA"):
        b2.linear(x, torch.zeros(3, 8))
    with pytest.raises(ValueError, match="CUDA"):
        b2.linear_grad(torch.zeros(4, 3), x, torch.zeros(3, 8))
    with pytest.raises(TypeError):
        b2.linear([1.0], w)


def central(f, x, h=1e-6):
    """df/dx for a scalar f, an element at a time."""
    g = torch.empty_like(x)
    for i in range(x.numel()):
        e = torch.zeros_like(x).view(-1)
        e[i] = h
        e = e.view(x.shape)
        g.view(-1)[i] = (f(x + e) - f(x - e)) / (2 * h)
    return g


def test_layer_formula_against_differences():
    gen = torch.Generator().manual_seed(0)
    r = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    s, g, b, dy, ds = r(3, 6), r(6), r(6), r(3, 6), r(3, 6)
    _, mean, inv, _ = F.layer(s, g, b, 1e-5)
    (dx, dg, db, dc), _ = F.layer_grad(dy, s, mean, inv, g, ds)

    def loss(sv, gv, bv):
        return (dy * F.layer(sv, gv, bv, 1e-5)[0]).sum() + (ds * sv).sum()
    torch.testing.assert_close(dx, central(lambda v: loss(v, g, b), s), rtol=1e-6, atol=1e-7)
    torch.testing.assert_close(dg, central(lambda v: loss(s, v, b), g), rtol=1e-6, atol=1e-7)
    torch.testing.assert_close(db, central(lambda v: loss(s, g, v), b), rtol=1e-6, atol=1e-7)
    torch.testing.assert_close(dc, central(lambda v: loss(s + v, g, b), torch.zeros_like(b)),
                               rtol=1e-6, atol=1e-7)


@pytest.mark.parametrize("name", sorted(F.ACTIVATIONS))
def test_linear_formula_against_differences(name):
    gen = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    x, w, b, dy = r(3, 4), r(5, 4), r(5), r(3, 5)
    z = x @ w.t() + b
    (dx, dw, db), _ = F.linear_grad(dy, x, w, z, name)

    def loss(xv, wv, bv):
        return (dy * F.linear(xv, wv, bv, None, name)[0][0]).sum()
    torch.testing.assert_close(dx, central(lambda v: loss(v, w, b), x), rtol=1e-6, atol=1e-7)
    torch.testing.assert_close(dw, central(lambda v: loss(x, v, b), w), rtol=1e-6, atol=1e-7)
    torch.testing.assert_close(db, central(lambda v: loss(x, w, v), b), rtol=1e-6, atol=1e-7)

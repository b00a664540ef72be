"""GPU: the linear operator at sizes where a kernel does everything more than once:
several tiles per CTA in every layout, over 32 parts of the bias gradient, the large
float32 tile with its ring of slices reused.

With whole numbers all products are whole and every partial sum is below 2^24, so
that binary32 holds it exactly in any order: a slice, row or tile that is left out,
taken twice or taken from another place changes the result.  Values with fractions
are held against the binary64 formulas."""
import pytest
import torch

import formulas as F
import residual_add_normalization_gb300 as b2
from test_linear import check_forward, check_grad, dev, make

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _no_wait_gave_up():
    yield
    b2.library().b200norm_testing_force_linear(0, 0, 0, 0)
    b2.linear_status()


def whole(shape, t, seed, shift):
    """Whole numbers from -2 to 2, starting `shift` elements into their block."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    return dev(torch.randint(-2, 3, shape, generator=g, device="cuda", dtype=torch.int8).to(t),
               shift)


def check_exact(rows, n_in, n_out, t, relu=False, shift=0):
    x, w, bias, residual, dy = (whole(s, t, i, shift) for i, s in enumerate(
        ((rows, n_in), (n_out, n_in), (n_out,), (rows, n_out), (rows, n_out))))
    z64 = x.double() @ w.double().t() + bias.double()
    y64 = (z64.clamp(min=0) if relu else z64) + residual.double()
    y, z = b2.linear(x, w, bias, residual, activation=4 if relu else 0, want_z=True)
    assert torch.equal(z, z64.to(t)) and torch.equal(y, y64.to(t))
    d64 = dy.double() * (z.double() > 0) if relu else dy.double()
    dx, dw, db = b2.linear_grad(dy, x, w, z, activation=4 if relu else 0)
    assert torch.equal(dx, (d64 @ w.double()).to(t))
    assert torch.equal(dw, (d64.t() @ x.double()).to(t))
    assert torch.equal(db, d64.sum(0).to(t))


TILINGS = [(2, 256), (1, 128), (1, 64)]
# tiles of 256 x 256: of y 198, of dW 198, of dx 198 (76 pairs of CTAs at most)
WIDE = [(2600, 136, 4360), (136, 2600, 4360), (2600, 4360, 136)]


@pytest.mark.parametrize("t", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("shape", WIDE)
@pytest.mark.parametrize("tiling", TILINGS)
def test_several_tiles_per_cta(tiling, shape, t):
    assert b2.library().b200norm_testing_force_linear(*tiling, 1, 0) == 0
    for relu in (False, True):
        check_exact(*shape, t, relu)


@pytest.mark.parametrize("t", ["bf16", "f16"])
@pytest.mark.parametrize("name", ["gelu", "silu"])
@pytest.mark.parametrize("tiling", TILINGS)
def test_several_tiles_per_cta_with_everything(tiling, name, t):
    """z kept, residual and activation at once, on values with fractions."""
    assert b2.library().b200norm_testing_force_linear(*tiling, 1, 0) == 0
    check_forward(make(2600, 136, 4360, t, 15), name, True, True, True)


@pytest.mark.parametrize("t", ["bf16", "f16"])
@pytest.mark.parametrize("shape", WIDE)
def test_grad_of_many_tiles(shape, t):
    check_grad(make(*shape, t, 16), "gelu")


@pytest.mark.parametrize("t", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("shape", [(4500, 72, 40), (16384, 520, 264), (40000, 16, 24),
                                   (9001, 264, 136)])
def test_many_rows(shape, t):
    """Long sums over rows: over 32 parts of db, dW's K of up to 40,000."""
    for relu in (False, True):
        check_exact(*shape, t, relu)


@pytest.mark.parametrize("shape,shift", [((4501, 71, 41), 0), ((2000, 1027, 515), 0),
                                         ((2000, 264, 520), 1)])
@pytest.mark.parametrize("t", [torch.bfloat16, torch.float16, torch.float32])
def test_many_rows_that_are_not_whole_vectors(shape, shift, t):
    for relu in (False, True):
        check_exact(*shape, t, relu, shift)


# at least 128 tiles of 128 x 128 in y, dx and dW: whole vectors, ragged, unaligned
LARGE_F32 = [((1536, 1408, 1664), 0), ((1500, 1411, 1530), 0), ((1536, 1408, 1664), 1),
             ((1665, 1444, 1412), 0)]


@pytest.mark.parametrize("shape,shift", LARGE_F32)
def test_large_float32_exact(shape, shift):
    for relu in (False, True):
        check_exact(*shape, torch.float32, relu, shift)


@pytest.mark.parametrize("shape,shift", LARGE_F32)
@pytest.mark.parametrize("name", ["none", "gelu_tanh"])
def test_large_float32(name, shape, shift):
    d = make(*shape, "f32", 17)
    check_forward(d, name, True, name == "none", name != "none", shift)
    check_grad(d, name, shift)

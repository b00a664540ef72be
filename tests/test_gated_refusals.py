"""CPU: what the gated entry points refuse before any CUDA call, and the binary64 formulas
that the GPU tests use, against differentiation."""
import pytest
import torch

import gated_formulas as GF
import residual_add_normalization_gb300 as b2
from formulas import ACTIVATIONS
from residual_add_normalization_gb300 import buildlib

OK, INVALID, UNSUPPORTED, CUDA, WORKSPACE, TIMEOUT = range(6)
F32, F16, BF16 = 0, 1, 2
G = 1 << 30
FAKE = 1 << 40  # never dereferenced: every call below fails validation or is empty


@pytest.fixture(scope="module")
def lib():
    buildlib.build()
    return b2.library()


def gated(lib, **kw):
    a = dict(x=FAKE, w=FAKE + G, bias=None, h=FAKE + 3 * G, z=None, rows=4, n_in=64, n_out=32,
             T=F16, act=1, ws=None, wsb=0)
    a.update(kw)
    return lib.b200norm_gated_linear(*a.values(), None)


def test_forward_refusals(lib):
    assert gated(lib, T=3) == UNSUPPORTED
    assert gated(lib, rows=-1) == INVALID
    assert gated(lib, n_in=0) == INVALID
    assert gated(lib, n_out=0) == INVALID
    assert gated(lib, n_out=(1 << 19) + 1) == UNSUPPORTED
    assert gated(lib, n_in=(1 << 20) + 1) == UNSUPPORTED
    assert gated(lib, rows=(1 << 30) + 1) == UNSUPPORTED
    assert gated(lib, act=5) == INVALID
    assert gated(lib, act=-1) == INVALID
    assert gated(lib, x=None) == INVALID
    assert gated(lib, w=None) == INVALID
    assert gated(lib, h=None) == INVALID
    assert gated(lib, x=FAKE + 1) == INVALID
    assert gated(lib, h=FAKE) == INVALID                       # over x
    assert gated(lib, h=FAKE + G + 2 * 32 * 64 * 2 - 64) == INVALID  # over the weight's last row
    assert gated(lib, z=FAKE + 3 * G + 64) == INVALID          # over h
    assert gated(lib, bias=FAKE + 3 * G - 64) == INVALID       # its second half under h
    assert gated(lib, rows=5, n_in=63) == WORKSPACE                    # rows at no 16-byte boundary
    assert gated(lib, rows=5, n_in=63, ws=FAKE + 5 * G, wsb=100) == WORKSPACE
    assert gated(lib, rows=5, n_in=63, ws=FAKE + 5 * G + 8, wsb=1 << 20) == WORKSPACE
    assert gated(lib, rows=5, n_in=63, ws=FAKE + 3 * G, wsb=1 << 20) == WORKSPACE  # over h
    assert gated(lib, rows=0, x=None, w=None, h=None) == OK


def grad(lib, **kw):
    a = dict(dh=FAKE, x=FAKE + G, w=FAKE + 2 * G, z=FAKE + 3 * G, dx=FAKE + 4 * G,
             dw=FAKE + 5 * G, db=FAKE + 6 * G, rows=4, n_in=64, n_out=32, T=F16, act=1,
             ws=FAKE + 7 * G, wsb=1 << 20)
    a.update(kw)
    return lib.b200norm_gated_linear_grad(*a.values(), None)


def test_gradient_refusals(lib):
    assert grad(lib, T=3) == UNSUPPORTED
    assert grad(lib, n_out=(1 << 19) + 1) == UNSUPPORTED
    assert grad(lib, act=9) == INVALID
    for name in ("dh", "x", "w", "z"):
        assert grad(lib, **{name: None}) == INVALID, name
        assert grad(lib, **{name: FAKE + 9 * G + 1}) == INVALID, name
    assert grad(lib, dx=FAKE + G) == INVALID
    assert grad(lib, dw=FAKE + 2 * G) == INVALID
    assert grad(lib, dw=FAKE + 3 * G + 64) == INVALID          # over z
    assert grad(lib, db=FAKE + 5 * G + 2 * 32 * 64 * 2 - 64) == INVALID  # over dw's last row
    assert grad(lib, ws=None) == WORKSPACE
    assert grad(lib, wsb=64) == WORKSPACE
    assert grad(lib, ws=FAKE + 7 * G + 128) == WORKSPACE
    assert grad(lib, ws=FAKE) == WORKSPACE
    assert grad(lib, dx=None, dw=None, db=None) == OK


def test_workspaces(lib):
    fw, bw = lib.b200norm_gated_linear_workspace_size, lib.b200norm_gated_linear_grad_workspace_size
    assert fw(100, 64, 32, F16, 1) == 0 and fw(100, 64, 31, F32, 0) == 0
    # both operands in rows of 72 elements, each from a 256-byte boundary
    assert fw(100, 65, 32, F16, 1) == -(-100 * 72 * 2 // 256) * 256 + -(-64 * 72 * 2 // 256) * 256
    assert fw(100, 64, 32, F16, 0) > 0
    assert bw(100, 64, 32, F16, 1) >= 100 * 64 * 2 + 64 * 4  # dz, and a part of the sums
    assert fw(-1, 64, 32, F16, 1) == 0 and bw(4, 64, 1 << 20, F16, 1) == 0


def test_python_refusals():
    with pytest.raises(ValueError, match="no CPU path"):
        b2.gated_linear(torch.zeros(2, 4), torch.zeros(6, 4))


@pytest.mark.gpu
def test_python_refusals_of_cuda_tensors():
    x, w, z, h = (torch.zeros(s, device="cuda") for s in ((3, 8), (12, 8), (3, 12), (3, 6)))
    bad = [(ValueError, lambda: b2.gated_linear(x, w[:11])),
           (ValueError, lambda: b2.gated_linear(x[:, :4].contiguous(), w)),
           (ValueError, lambda: b2.gated_linear(x, w, w[0])),
           (ValueError, lambda: b2.gated_linear(x, w.t())),
           (TypeError, lambda: b2.gated_linear(x, w.half())),
           (ValueError, lambda: b2.gated_linear(x, w, h=z)),
           (ValueError, lambda: b2.gated_linear(x, w, z=h)),
           (b2.B200NormError, lambda: b2.gated_linear(x, w, activation=7)),
           (ValueError, lambda: b2.gated_linear_grad(z, x, w, z)),
           (ValueError, lambda: b2.gated_linear_grad(h, x, w, h)),
           (ValueError, lambda: b2.gated_linear_grad(h, h, w, z)),
           (TypeError, lambda: b2.gated_linear_grad(h, x, w, None)),
           (ValueError, lambda: b2.gated_linear_grad(h, x, w, z, db=h)),
           (b2.B200NormError, lambda: b2.gated_linear_grad(h, x, w, z, dx=x))]
    for i, (kind, call) in enumerate(bad):
        with pytest.raises(kind):
            call()
            pytest.fail(f"call {i} was taken")


@pytest.mark.parametrize("act", sorted(ACTIVATIONS))
def test_formulas_against_differentiation(act):
    gen = torch.Generator().manual_seed(1)
    x, w, b, dh = (torch.randn(s, generator=gen, dtype=torch.float64)
                   for s in ((5, 7), (12, 7), (12,), (5, 6)))
    for v in (x, w, b):
        v.requires_grad_()
    (h, z), _ = GF.gated(x, w, b, act)
    h.backward(dh)
    ref, _ = GF.gated_grad(dh, x.detach(), w.detach(), z.detach(), act)
    for got, want in zip(ref, (x.grad, w.grad, b.grad)):
        assert torch.allclose(got, want, rtol=1e-11, atol=1e-12)

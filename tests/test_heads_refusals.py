"""CPU: what the head entry points refuse before any CUDA call, their frequencies, and the
binary64 formulas that the GPU tests use, against differentiation."""
import ctypes
import math

import pytest
import torch

import head_formulas as H
import residual_add_normalization_gb300 as b2
from residual_add_normalization_gb300 import buildlib

OK, INVALID, UNSUPPORTED, CUDA, WORKSPACE, TIMEOUT = range(6)
F32, F16, BF16 = 0, 1, 2
G = 1 << 30
FAKE = 1 << 40  # never dereferenced: every call below fails validation or is empty
I64 = (1 << 63) - 1


@pytest.fixture(scope="module")
def lib():
    buildlib.build()
    return b2.library()


def rotation(**kw):
    a = dict(positions=FAKE + 9 * G, bytes=8, sb=5, st=1, freq=FAKE + 10 * G, rot=64, inter=0,
             scale=1.0)
    a.update(kw)
    return b2._ROTATION.pack(*a.values())


def one(**kw):
    """Queries of (2, 5, 4, 64), dense."""
    a = dict(x=FAKE, y=FAKE + G, gamma=0, heads=4, xb=1280, xt=256, xh=64, yb=1280, yt=256, yh=64)
    a.update(kw)
    return b2._HEADS.pack(*a.values())


def keys(**kw):
    return one(**{**dict(x=FAKE + 2 * G, y=FAKE + 3 * G), **kw})


def norm(lib, q=None, k=None, r=None, batch=2, seq=5, size=64, T=F16, M=F16, eps=1e-6):
    return lib.b200norm_head_rms_rotary(q, k, rotation() if r is None else r, batch, seq, size, T,
                                        M, eps, None)


def rotary(lib, q=None, k=None, r=None, batch=2, seq=5, size=64, T=F16, inverse=0):
    return lib.b200norm_rotary(q, k, rotation() if r is None else r, batch, seq, size, T, inverse,
                               None)


def test_forward_refusals(lib):
    q = one()
    assert norm(lib, q, T=3, M=3) == UNSUPPORTED
    assert norm(lib, q, M=BF16) == UNSUPPORTED
    assert norm(lib, q, T=F32, M=F16) == UNSUPPORTED
    assert norm(lib, q, batch=-1) == INVALID
    assert norm(lib, q, size=0) == INVALID
    assert norm(lib, q, size=1025) == UNSUPPORTED
    assert norm(lib, one(heads=-1)) == INVALID
    assert norm(lib, one(heads=(1 << 16) + 1)) == UNSUPPORTED
    assert norm(lib, q, batch=1 << 16, seq=1 << 16) == UNSUPPORTED
    assert norm(lib, one(heads=1 << 12), batch=1 << 14, seq=1 << 15) == UNSUPPORTED
    assert norm(lib, q, eps=-1.0) == INVALID
    assert norm(lib, q, eps=float("nan")) == INVALID
    assert rotary(lib, q, inverse=2) == INVALID
    assert rotary(lib, one(gamma=FAKE + 5 * G)) == INVALID
    assert norm(lib, one(x=0)) == INVALID
    assert norm(lib, one(y=0)) == INVALID
    assert norm(lib, one(x=FAKE + 1)) == INVALID
    assert norm(lib, one(gamma=FAKE + 5 * G + 2), M=F32) == INVALID
    assert norm(lib, one(xt=-256)) == INVALID
    assert norm(lib, one(xb=I64)) == INVALID
    assert lib.b200norm_rotary(q, None, None, 2, 5, 64, F16, 0, None) == INVALID


def test_rotation_refusals(lib):
    q = one()
    for bad in (dict(rot=63), dict(rot=-2), dict(rot=66), dict(inter=2), dict(bytes=2),
                dict(positions=0), dict(freq=0), dict(positions=FAKE + 4), dict(freq=FAKE + 4),
                dict(sb=-1), dict(st=-1), dict(sb=I64), dict(scale=float("inf")),
                dict(scale=float("nan"))):
        assert norm(lib, q, r=rotation(**bad)) == INVALID, bad
        assert rotary(lib, q, r=rotation(**bad)) == INVALID, bad


def test_overlap_refusals(lib):
    assert rotary(lib, one(y=FAKE + 64)) == INVALID                       # over the input
    assert b"overlaps queries x" in lib.b200norm_last_error()
    assert rotary(lib, one(y=FAKE, yt=512)) == INVALID                    # in place, other steps
    assert rotary(lib, one(yt=0)) == INVALID                              # an element twice
    assert b"itself" in lib.b200norm_last_error()
    assert rotary(lib, one(yh=32)) == INVALID
    assert rotary(lib, one(yb=1000)) == INVALID
    assert rotary(lib, one(), keys(y=FAKE + G)) == INVALID                # over the other result
    assert rotary(lib, one(), keys(y=FAKE)) == INVALID                    # over the other input
    assert rotary(lib, one(y=FAKE + 9 * G)) == INVALID                    # over the positions
    assert rotary(lib, one(y=FAKE + 10 * G)) == INVALID                   # over the frequencies
    assert norm(lib, one(gamma=FAKE + G + 128)) == INVALID                # over gamma
    # side by side in one row, but one too many
    wide = dict(yb=3840, yt=768)
    assert rotary(lib, one(y=FAKE + G, **wide), keys(y=FAKE + G + 2 * 192, **wide)) == INVALID
    assert b"outputs overlap" in lib.b200norm_last_error()


def test_overlap_refusals_of_heads_that_alternate(lib):
    """Queries and keys head by head in rows of 4 x 128: one element into the other's place."""
    apart = dict(yb=2560, yt=512, yh=128)
    for at in (63 * 2, 65 * 2, 127 * 2, (512 + 1) * 2):
        assert rotary(lib, one(y=FAKE + G, **apart), keys(y=FAKE + G + at, **apart)) == INVALID, at
        assert b"outputs overlap" in lib.b200norm_last_error()
    # steps that are not each other's multiples
    assert rotary(lib, one(y=FAKE + G, **apart),
                  keys(y=FAKE + G + 128, **{**apart, "yh": 192})) == INVALID


def test_empty_calls_do_nothing(lib):
    none = one(x=0, y=0)
    assert norm(lib, none, batch=0) == OK
    assert norm(lib, none, seq=0, r=rotation(positions=0, freq=0)) == OK
    assert norm(lib, one(x=0, y=0, heads=0)) == OK
    assert norm(lib) == OK
    assert rotary(lib, none, seq=0) == OK


def grad_set(**kw):
    a = dict(dy=FAKE, x=FAKE + G, gamma=FAKE + 5 * G, dx=FAKE + 2 * G, dgamma=FAKE + 6 * G,
             heads=4, db=1280, dt=256, dh=64, xb=1280, xt=256, xh=64, yb=1280, yt=256, yh=64)
    a.update(kw)
    return b2._HEADS_GRAD.pack(*a.values())


def grad(lib, q=None, k=None, r=None, batch=2, seq=5, size=64, T=F16, M=F16, eps=1e-6,
         ws=FAKE + 8 * G, wsb=1 << 20):
    return lib.b200norm_head_rms_rotary_grad(q, k, rotation() if r is None else r, batch, seq,
                                             size, T, M, eps, ws, wsb, None)


def test_gradient_refusals(lib):
    q = grad_set()
    assert grad(lib, q, T=3, M=3) == UNSUPPORTED
    assert grad(lib, q, M=BF16) == UNSUPPORTED
    assert grad(lib, q, size=1025) == UNSUPPORTED
    assert grad(lib, q, eps=-1.0) == INVALID
    assert grad(lib, q, r=rotation(rot=63)) == INVALID
    assert grad(lib, grad_set(dy=0)) == INVALID
    assert grad(lib, grad_set(x=0)) == INVALID
    assert grad(lib, grad_set(x=FAKE + G + 1)) == INVALID
    assert grad(lib, grad_set(gamma=FAKE + 5 * G + 1)) == INVALID
    assert grad(lib, grad_set(dgamma=FAKE + 6 * G + 1)) == INVALID
    assert grad(lib, grad_set(dx=FAKE)) == INVALID                        # over dy
    assert grad(lib, grad_set(dx=FAKE + G)) == INVALID                    # over x
    assert grad(lib, grad_set(dx=FAKE + 5 * G)) == INVALID                # over gamma
    assert grad(lib, grad_set(dgamma=FAKE + 2 * G + 64)) == INVALID       # over dx
    assert grad(lib, grad_set(dgamma=FAKE + 64)) == INVALID               # over dy
    assert grad(lib, grad_set(dgamma=FAKE + 5 * G)) == INVALID            # over gamma
    assert grad(lib, grad_set(yt=0)) == INVALID                           # an element twice
    assert grad(lib, q, grad_set(dx=FAKE + 4 * G)) == INVALID             # one dgamma for both
    assert grad(lib, q, grad_set(dgamma=FAKE + 7 * G)) == INVALID         # one dx for both
    assert grad(lib, q, ws=None) == WORKSPACE
    assert grad(lib, q, wsb=16) == WORKSPACE
    assert grad(lib, q, ws=FAKE + 8 * G + 64) == WORKSPACE
    assert grad(lib, q, ws=FAKE) == WORKSPACE                             # over dy
    assert grad(lib, q, ws=FAKE + 5 * G) == WORKSPACE                     # over gamma
    assert grad(lib, grad_set(dx=0, dgamma=0)) == OK                      # nothing wanted
    assert grad(lib, grad_set(heads=0)) == OK


def test_gradient_workspace_covers_a_call_of_one_tensor(lib):
    """Sized for both tensors, it serves a call that wants one tensor's gradients."""
    size = lib.b200norm_head_rms_rotary_grad_workspace_size
    for tokens in (1, 2, 7, 100, 5000, 100000):
        for q in (1, 3, 8, 32):
            for k in (1, 2, 8):
                both = size(1, tokens, q, k, 128)
                assert both >= size(1, tokens, q, 0, 128) > 0
                assert both >= size(1, tokens, 0, k, 128) > 0
    assert size(0, 4, 2, 2, 64) == 0 and size(1, 4, 0, 0, 64) == 0 and size(1, 4, 2, 2, 0) == 0


def test_python_refusals():
    x = torch.zeros(4, 2, 8)
    p, f = torch.zeros(4, dtype=torch.int64), torch.zeros(4, dtype=torch.float64)
    with pytest.raises(ValueError, match="no CPU path"):
        b2.rotary(x, None, p, f)
    with pytest.raises(ValueError, match="queries or keys"):
        b2.rotary(None, None, p, f)
    with pytest.raises(TypeError, match="torch.Tensor"):
        b2.head_rms_rotary([1.0], None, None, None, p, f)


@pytest.mark.gpu
def test_python_refusals_of_cuda_tensors():
    x = torch.zeros(4, 2, 8, device="cuda")
    p = torch.zeros(4, dtype=torch.int64, device="cuda")
    f = torch.zeros(4, dtype=torch.float64, device="cuda")
    g = torch.ones(8, device="cuda")
    bad = [(ValueError, lambda: b2.rotary(x[0], None, p, f)),
           (ValueError, lambda: b2.rotary(x, x[:3], p, f)),
           (ValueError, lambda: b2.rotary(x, x[..., :4], p, f)),
           (ValueError, lambda: b2.rotary(x.transpose(1, 2), None, p, f)),
           (TypeError, lambda: b2.rotary(x, x.half(), p, f)),
           (TypeError, lambda: b2.rotary(x.double(), None, p, f)),
           (ValueError, lambda: b2.rotary(x, None, p[:3], f)),
           (TypeError, lambda: b2.rotary(x, None, p.float(), f)),
           (TypeError, lambda: b2.rotary(x, None, None, f)),
           (TypeError, lambda: b2.rotary(x, None, p, f.float())),
           (ValueError, lambda: b2.rotary(x, None, p, None)),
           (ValueError, lambda: b2.rotary(x, None, p, f.cpu())),
           (ValueError, lambda: b2.rotary(x, None, p.cpu(), f)),
           (ValueError, lambda: b2.rotary(x, None, p, f[::2])),
           (b2.B200NormError, lambda: b2.rotary(x, None, p, torch.cat((f, f)))),
           (ValueError, lambda: b2.rotary(x, None, p, f, q_out=x[:, :1])),
           (ValueError, lambda: b2.rotary(x, None, p, f, k_out=x)),
           (b2.B200NormError, lambda: b2.rotary(x, None, p, f, q_out=x[:1].expand(4, 2, 8))),
           (b2.B200NormError, lambda: b2.rotary(x[:, :1], None, p, f, q_out=x[:, 1:].transpose(0, 1)
                                                .transpose(0, 1).as_strided((4, 1, 8), (8, 8, 1)))),
           (ValueError, lambda: b2.head_rms_rotary(x, None, g[:4], None, p, f)),
           (TypeError, lambda: b2.head_rms_rotary(x, None, g.half(), None, p, f)),
           (ValueError, lambda: b2.head_rms_rotary(x, None, None, g, p, f)),
           (TypeError, lambda: b2.head_rms_rotary(x.half(), x.half(), g, g.half(), p, f)),
           (b2.B200NormError, lambda: b2.head_rms_rotary(x, None, g, None, p, f, epsilon=-1.0)),
           (TypeError, lambda: b2.head_rms_rotary_grad(None, None, x, None, g, None, p, f)),
           (ValueError, lambda: b2.head_rms_rotary_grad(x[:3], None, x, None, g, None, p, f)),
           (ValueError, lambda: b2.head_rms_rotary_grad(x, x, x, None, g, None, p, f)),
           (ValueError, lambda: b2.head_rms_rotary_grad(x, None, x, None, None, None, p, f,
                                                        dgamma_q=g)),
           (b2.B200NormError, lambda: b2.head_rms_rotary_grad(x, None, x, None, g, None, p, f,
                                                              dq_out=x))]
    for i, (kind, call) in enumerate(bad):
        with pytest.raises(kind):
            call()
            pytest.fail(f"call {i} was taken")


@pytest.mark.gpu
@pytest.mark.parametrize("wrong", [[1.0] * 8, 1.0, "ones"])
def test_gammas_that_are_no_tensors(wrong):
    x = torch.zeros(4, 2, 8, device="cuda")
    p = torch.zeros(4, dtype=torch.int64, device="cuda")
    f = torch.zeros(4, dtype=torch.float64, device="cuda")
    g = torch.ones(8, device="cuda")
    for gq, gk in ((wrong, g), (g, wrong), (wrong, wrong)):
        with pytest.raises(TypeError, match="torch.Tensor"):
            b2.head_rms_rotary(x, x, gq, gk, p, f)
        with pytest.raises(TypeError, match="torch.Tensor"):
            b2.head_rms_rotary_grad(x, x, x, x, gq, gk, p, f)


def freqs(lib, n, base=10000.0, scaling=0, factor=1.0, length=0.0, low=1.0, high=32.0):
    out = (ctypes.c_double * (max(n, 2) // 2))()
    st = lib.b200norm_rotary_frequencies(out, n, base, scaling, factor, length, low, high)
    return list(out) if st == OK else st


def test_frequencies(lib):
    plain = freqs(lib, 64)
    for i, f in enumerate(plain):
        assert abs(f - 10000.0 ** (-i / 32)) <= 1e-15 * f
    assert freqs(lib, 64, scaling=1, factor=4.0) == [f / 4.0 for f in plain]
    based = freqs(lib, 64, scaling=2, factor=8.0)
    assert based[0] == 1.0 and abs(based[-1] - plain[-1] / 8) <= 1e-14 * plain[-1]
    for i, f in enumerate(based):
        assert abs(f / plain[i] - 8.0 ** (-i / 31)) <= 1e-13
    turns = freqs(lib, 64, scaling=3, factor=8.0, length=8192.0, low=1.0, high=32.0)
    for f, g in zip(plain, turns):
        t = 8192 * f / (2 * math.pi)
        if t >= 32:
            assert g == f
        elif t <= 1:
            assert abs(g - f / 8) <= 1e-15 * f
        else:
            w = (t - 1) / 31
            assert abs(g - (f * w + f / 8 * (1 - w))) <= 1e-14 * f
    assert any(1 < 8192 * f / (2 * math.pi) < 32 for f in plain)
    assert freqs(lib, 2) == [1.0]


def test_frequency_refusals(lib):
    for bad in (dict(n=0), dict(n=3), dict(n=1026), dict(n=64, base=0.0),
                dict(n=64, base=float("inf")), dict(n=64, scaling=4), dict(n=64, scaling=-1),
                dict(n=64, scaling=1, factor=0.0), dict(n=64, scaling=1, factor=float("nan")),
                dict(n=2, scaling=2, factor=2.0), dict(n=64, scaling=3, factor=2.0, length=0.0),
                dict(n=64, scaling=3, factor=2.0, length=8.0, low=2.0, high=2.0),
                dict(n=64, scaling=3, factor=2.0, length=8.0, low=-1.0)):
        assert freqs(lib, **bad) == INVALID, bad
    assert lib.b200norm_rotary_frequencies(None, 64, 10000.0, 0, 1.0, 0.0, 1.0, 32.0) == INVALID
    with pytest.raises(b2.B200NormError):
        b2.rotary_frequencies(7, device="cpu")
    got = b2.rotary_frequencies(64, scaling=b2.ROTARY_SCALINGS["linear"], factor=2.0, device="cpu")
    assert got.dtype is torch.float64 and got.tolist() == freqs(lib, 64, scaling=1, factor=2.0)


@pytest.mark.parametrize("interleaved", [False, True])
def test_formulas_against_differentiation(interleaved):
    gen = torch.Generator().manual_seed(1)
    x, dy = (torch.randn(2, 3, 4, 10, generator=gen, dtype=torch.float64) for _ in range(2))
    gamma = torch.randn(10, generator=gen, dtype=torch.float64)
    p = torch.tensor([[0, 5, 9], [100, 3, 70000]])
    turn = H.turn_of(p, torch.tensor([1.0, 0.1, 0.01, 0.001], dtype=torch.float64), 1.3)
    x.requires_grad_()
    gamma.requires_grad_()
    y, _ = H.head_norm(x, gamma, turn, 1e-6, interleaved)
    y.backward(dy)
    (dx, dg), _ = H.head_norm_grad(dy, x.detach(), gamma.detach(), turn, 1e-6, interleaved)
    assert torch.allclose(dx, x.grad, rtol=1e-12, atol=1e-13)
    assert torch.allclose(dg, gamma.grad, rtol=1e-12, atol=1e-13)
    back, _ = H.rotary(H.rotary(x.detach(), turn, interleaved)[0], turn.conj(), interleaved)
    assert torch.allclose(back[..., :8], x.detach()[..., :8] * 1.69, rtol=1e-12)

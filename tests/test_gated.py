"""GPU: the gated linear operator and its gradients against binary64."""
import time

import pytest
import torch

import gated_formulas as G
import residual_add_normalization_gb300 as b2
from formulas import ACTIVATIONS, DTYPES, assert_within

pytestmark = pytest.mark.gpu

TIMEOUT = 5


@pytest.fixture(autouse=True)
def _status():
    yield
    lib = b2.library()
    lib.b200norm_testing_force_linear(0, 0, 0, 0)
    lib.b200norm_testing_linear_stall(0, 0)
    b2.linear_status()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def tensor(g, shape, t, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(t)


def at_odd(t):
    """The same values one element past a boundary."""
    base = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
    base[1:] = t.flatten()
    return base[1:].view(t.shape)


def check_forward(rows, n_in, n_out, t, act="silu", bias=True, want_z=True, odd=False, seed=1):
    g = gen(seed)
    x, w = tensor(g, (rows, n_in), t), tensor(g, (2 * n_out, n_in), t, n_in ** -0.5)
    b = tensor(g, (2 * n_out,), t, 0.5) if bias else None
    if odd:
        x, w = at_odd(x), at_odd(w)
    h, z = b2.gated_linear(x, w, b, activation=ACTIVATIONS[act], want_z=want_z)
    (rh, rz), (eh, ez) = G.gated(x.cpu(), w.cpu(), None if b is None else b.cpu(), act)
    assert_within(h, rh, eh, "h")
    assert (z is None) == (not want_z)
    if want_z:
        assert_within(z, rz, ez, "z")
        # h does not depend on whether z is wanted
        assert torch.equal(b2.gated_linear(x, w, b, activation=ACTIVATIONS[act])[0], h)


@pytest.mark.parametrize("t", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,n_in,n_out", [
    (1, 1, 1), (1, 64, 8), (1, 768, 768), (2, 300, 33), (3, 512, 40), (4, 4096, 64),
    (5, 200, 72), (6, 516, 41), (8, 1024, 257), (16, 512, 100),
    (17, 1027, 130), (33, 256, 264), (64, 512, 512),
    (65, 128, 72), (129, 64, 200), (130, 96, 1000), (300, 520, 1027), (777, 136, 96)])
def test_forward(rows, n_in, n_out, t):
    check_forward(rows, n_in, n_out, DTYPES[t], bias=rows % 2 == 1, want_z=True)


@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("act", sorted(ACTIVATIONS))
@pytest.mark.parametrize("rows,n_in,n_out", [(1, 256, 64), (9, 320, 96), (200, 320, 200)])
def test_activations(rows, n_in, n_out, act, t):
    check_forward(rows, n_in, n_out, DTYPES[t], act=act, want_z=rows == 9)


@pytest.mark.parametrize("t", ["bf16", "f16"])
@pytest.mark.parametrize("rows,n_in,n_out", [(1, 256, 64), (2, 1000, 3000), (40, 264, 72),
                                             (300, 72, 136)])
def test_operands_at_odd_places(rows, n_in, n_out, t):
    check_forward(rows, n_in, n_out, DTYPES[t], odd=True)


@pytest.mark.parametrize("rows", [2, 4, 5, 6, 8, 9])
@pytest.mark.parametrize("n_in,n_out", [(256, 70), (258, 64), (4096, 3300)])
def test_float32_at_odd_places(rows, n_in, n_out):
    check_forward(rows, n_in, n_out, torch.float32, odd=True, bias=rows % 2 == 0)


TILINGS = ([(2, 256, 1, 0)] + [(1, 128, s, 0) for s in (1, 2, 4, 8)]
           + [(1, bn, s, 1) for bn in (16, 32, 64) for s in (1, 2, 4, 8)])


@pytest.mark.parametrize("tiling", TILINGS)
@pytest.mark.parametrize("rows,n_in,n_out", [(16, 520, 8), (13, 576, 64), (11, 1000, 300),
                                             (16, 512, 1096), (7, 640, 131)])
def test_every_tiling(rows, n_in, n_out, tiling):
    """Edges of each tiling: the gate's last columns lie next to what it gates, and must not
    reach it.  (The results of 131 columns are not whole vectors.)"""
    assert b2.library().b200norm_testing_force_linear(*tiling) == 0
    check_forward(rows, n_in, n_out, torch.bfloat16, seed=3)
    check_forward(rows, n_in, n_out, torch.float16, bias=False, want_z=False, seed=4)


@pytest.mark.parametrize("tiling", [(2, 256, 1, 0), (1, 128, 1, 0)])
@pytest.mark.parametrize("rows,n_in,n_out", [(2100, 128, 2056), (1500, 72, 3001)])
def test_many_tiles(rows, n_in, n_out, tiling):
    """Several tiles a CTA: both buffers of sums and of results come round again.  In whole
    numbers, exactly: x and w in {-1, 0, 1}, no activation, |z| at most 128."""
    assert b2.library().b200norm_testing_force_linear(*tiling) == 0
    g = gen(5)
    x, w = (torch.randint(-1, 2, s, generator=g, device="cuda").half()
            for s in ((rows, n_in), (2 * n_out, n_in)))
    want = x.float() @ w.float().t()
    for want_z in (True, False):
        h, z = b2.gated_linear(x, w, activation=0, want_z=want_z)
        assert torch.equal(h, (want[:, :n_out] * want[:, n_out:]).half())
        if want_z:
            assert torch.equal(z, want.half())


def test_a_tiling_without_a_kernel_is_refused():
    x, w = (torch.ones(s, device="cuda").bfloat16() for s in ((40, 64), (128, 64)))
    for tiling in ((1, 64, 1, 0), (1, 16, 1, 1), (2, 256, 2, 0)):
        assert b2.library().b200norm_testing_force_linear(*tiling) == 0
        with pytest.raises(b2.B200NormError):
            b2.gated_linear(x, w)


@pytest.mark.parametrize("t", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("rows,n_in,n_out", [(1, 64, 8), (3, 100, 33), (64, 128, 72),
                                             (130, 256, 320), (333, 77, 131)])
def test_gradient(rows, n_in, n_out, act, t):
    g = gen(6)
    x, w = tensor(g, (rows, n_in), DTYPES[t]), tensor(g, (2 * n_out, n_in), DTYPES[t], n_in ** -0.5)
    dh, z = tensor(g, (rows, n_out), DTYPES[t], 0.3), tensor(g, (rows, 2 * n_out), DTYPES[t], 2.0)
    got = b2.gated_linear_grad(dh, x, w, z, activation=ACTIVATIONS[act])
    ref, bound = G.gated_grad(dh.cpu(), x.cpu(), w.cpu(), z.cpu(), act)
    for a, r, e, name in zip(got, ref, bound, ("dx", "dw", "db")):
        assert_within(a, r, e, name)
    for i, one in enumerate((dict(want_weight=False, want_bias=False),
                             dict(want_input=False, want_bias=False),
                             dict(want_input=False, want_weight=False))):
        alone = b2.gated_linear_grad(dh, x, w, z, activation=ACTIVATIONS[act], **one)
        assert torch.equal(alone[i], got[i])
        assert sum(v is not None for v in alone) == 1


@pytest.mark.parametrize("t", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("odd", [False, True])
@pytest.mark.parametrize("rows,n_in,n_out", [
    (1, 1, 1), (1, 4096, 600), (2, 256, 17), (2, 30, 300), (3, 264, 40), (4, 129, 65),
    (5, 516, 130), (7, 64, 1000), (8, 1024, 333), (8, 33, 8), (9, 264, 40)])
def test_gradient_of_few_rows(rows, n_in, n_out, odd, t):
    """The weight, x and the weight's gradient at and off 16-byte boundaries; every part of the
    result by itself and into given tensors, with what lies around them left alone."""
    act = sorted(ACTIVATIONS)[rows % 5]
    g = gen(31)
    x, w = tensor(g, (rows, n_in), DTYPES[t]), tensor(g, (2 * n_out, n_in), DTYPES[t], n_in ** -0.5)
    dh, z = tensor(g, (rows, n_out), DTYPES[t], 0.3), tensor(g, (rows, 2 * n_out), DTYPES[t], 2.0)
    if odd:
        x, w, dh, z = at_odd(x), at_odd(w), at_odd(dh), at_odd(z)
    code, at = ACTIVATIONS[act], 1 if odd else 8
    shapes = (x.shape, w.shape, (2 * n_out,))
    bases = [torch.full((at + torch.Size(s).numel() + 8,), 7.0, dtype=DTYPES[t], device="cuda")
             for s in shapes]
    into = [b[at:-8].view(s) for b, s in zip(bases, shapes)]
    got = b2.gated_linear_grad(dh, x, w, z, activation=code, dx=into[0], dw=into[1], db=into[2])
    ref, bound = G.gated_grad(dh.cpu(), x.cpu(), w.cpu(), z.cpu(), act)
    for a, r, e, name in zip(got, ref, bound, ("dx", "dw", "db")):
        assert_within(a, r, e, name)
    assert all(bool((b[:at] == 7).all()) and bool((b[-8:] == 7).all()) for b in bases)
    for i, one in enumerate((dict(want_weight=False, want_bias=False),
                             dict(want_input=False, want_bias=False),
                             dict(want_input=False, want_weight=False))):
        assert torch.equal(b2.gated_linear_grad(dh, x, w, z, activation=code, **one)[i], got[i])


def test_gradient_of_few_rows_stays_in_its_row():
    """NaN and infinities of one row: dx of the others is as it was, though rows share
    registers."""
    g = gen(32)
    x, w = tensor(g, (3, 96), torch.bfloat16), tensor(g, (80, 96), torch.bfloat16)
    dh, z = tensor(g, (3, 40), torch.bfloat16), tensor(g, (3, 80), torch.bfloat16)
    want = b2.gated_linear_grad(dh, x, w, z)[0]
    dh[1, 5], z[1, 50] = float("nan"), float("inf")
    got = b2.gated_linear_grad(dh, x, w, z)
    assert torch.equal(got[0][::2], want[::2]) and bool(torch.isnan(got[0][1]).all())
    rows = torch.ones(80, dtype=torch.bool, device="cuda")
    rows[[5, 45, 10]] = False
    assert bool(torch.isfinite(got[1][rows].float()).all())
    assert not bool(torch.isfinite(got[1][~rows].float()).any())


@pytest.mark.parametrize("act", sorted(ACTIVATIONS))
def test_slopes(act):
    """dz element by element: a row a token, the weight a unit matrix, so that dx is dz's
    rows; over the whole range of gates."""
    n = 64
    gate = torch.cat((torch.linspace(-120, 120, 4001), torch.linspace(-6, 6, 4000)))
    rows = gate.numel() // 3
    g = gen(7)
    z = torch.randn(rows, 2 * n, generator=g, device="cuda")
    z[:, :3] = gate[:rows * 3].view(rows, 3).cuda()
    dh = torch.randn(rows, n, generator=g, device="cuda")
    w = torch.eye(2 * n, device="cuda")
    dx, _, _ = b2.gated_linear_grad(dh, w[:1].expand(rows, -1).contiguous(), w, z,
                                    activation=ACTIVATIONS[act], want_weight=False,
                                    want_bias=False)
    dz, e = G.dz_of(dh.cpu(), z.cpu(), act)
    assert_within(dx, dz, e, "dz")


def test_gradient_against_differences():
    g = gen(8)
    x, w = tensor(g, (3, 6), torch.float32), tensor(g, (10, 6), torch.float32)
    b, dh = tensor(g, (10,), torch.float32), tensor(g, (3, 5), torch.float32)
    h, z = b2.gated_linear(x, w, b, want_z=True)
    dx, dw, db = b2.gated_linear_grad(dh, x, w, z)
    args = [v.cpu().double() for v in (x, w, b)]

    def loss(v):
        return float((G.gated(*v, "silu")[0][0] * dh.cpu().double()).sum())
    step = 1e-5
    for which, got in enumerate((dx, dw, db)):
        for at in [(0,) * got.dim(), tuple(s - 1 for s in got.shape)]:
            up, down = [[v.clone() for v in args] for _ in range(2)]
            up[which][at] += step
            down[which][at] -= step
            want = (loss(up) - loss(down)) / (2 * step)
            assert abs(float(got[at]) - want) <= 1e-5 * (1 + abs(want))


def test_nothing_there():
    w = torch.ones(16, 8, device="cuda")
    x = torch.ones(0, 8, device="cuda")
    h, z = b2.gated_linear(x, w, want_z=True)
    assert h.shape == (0, 8) and z.shape == (0, 16)
    dx, dw, db = b2.gated_linear_grad(h, x, w, z)
    assert dx.shape == x.shape and bool((dw == 0).all()) and bool((db == 0).all())
    x3 = torch.randn(2, 3, 8, device="cuda")
    h, z = b2.gated_linear(x3, w, want_z=True)
    assert h.shape == (2, 3, 8) and z.shape == (2, 3, 16)
    assert b2.gated_linear_grad(h, x3, w, z)[0].shape == x3.shape


@pytest.mark.parametrize("rows", [1, 40, 300])
@pytest.mark.parametrize("t", ["bf16", "f32"])
def test_nan_stays_in_its_row_and_column(rows, t):
    g = gen(9)
    x, w = tensor(g, (rows, 200), DTYPES[t]), tensor(g, (240, 200), DTYPES[t], 0.1)
    clean, _ = b2.gated_linear(x, w)
    bad = w.clone()
    bad[7, 3] = float("nan")        # a gate's row
    bad[120 + 50, 9] = float("inf")  # a row of what it gates
    h, _ = b2.gated_linear(x, bad)
    keep = [i for i in range(120) if i not in (7, 50)]
    assert torch.equal(h[:, keep], clean[:, keep])
    assert bool(torch.isnan(h[:, 7]).all()) and not bool(torch.isfinite(h[:, 50]).any())
    if rows > 1:
        xb = x.clone()
        xb[rows // 2, 0] = float("nan")
        h, _ = b2.gated_linear(xb, w)
        rest = torch.arange(rows) != rows // 2
        assert torch.equal(h[rest.cuda()], clean[rest.cuda()])
        assert bool(torch.isnan(h[rows // 2]).all())


def test_equal_calls_give_equal_bits():
    g = gen(10)
    for rows, n_in, n_out, t in ((1, 4096, 512, "bf16"), (300, 1024, 520, "bf16"),
                                 (50, 512, 300, "f32"), (4000, 320, 264, "f16")):
        x, w = tensor(g, (rows, n_in), DTYPES[t]), tensor(g, (2 * n_out, n_in), DTYPES[t], 0.05)
        first = b2.gated_linear(x, w, want_z=True)
        grads = b2.gated_linear_grad(first[0], x, w, first[1])
        for _ in range(3):
            again = b2.gated_linear(x, w, want_z=True)
            assert all(torch.equal(a, b) for a, b in zip(first, again))
            assert all(torch.equal(a, b) for a, b in
                       zip(grads, b2.gated_linear_grad(first[0], x, w, first[1])))


@pytest.mark.parametrize("tiling", [(2, 256, 1, 0), (1, 128, 1, 0), (1, 128, 4, 0), (1, 16, 1, 1),
                                    (1, 16, 2, 1)])
def test_waits_give_up(tiling):
    """With nothing copied, the roles' waits run out: the call returns, the status says so
    once, and the next call is right."""
    lib = b2.library()
    g = gen(11)
    x, w = tensor(g, (16, 1024), torch.bfloat16), tensor(g, (600, 1024), torch.bfloat16)
    assert lib.b200norm_testing_force_linear(*tiling) == 0
    want, _ = b2.gated_linear(x, w)
    b2.linear_status()
    assert lib.b200norm_testing_linear_stall(1, 20_000_000) == 0
    t0 = time.monotonic()
    b2.gated_linear(x, w)
    with pytest.raises(b2.B200NormError) as e:
        b2.linear_status()
    assert e.value.status == TIMEOUT and time.monotonic() - t0 < 2.0
    assert lib.b200norm_testing_linear_stall(0, 0) == 0
    assert torch.equal(b2.gated_linear(x, w)[0], want)


def test_captured_and_replayed():
    """Two graphs, with scratch of their own (operands that are copied to aligned rows), give
    the eager call's bits with new inputs."""
    g = gen(12)
    x, w = tensor(g, (50, 131), torch.float16), tensor(g, (2 * 67, 131), torch.float16, 0.1)
    b2.gated_linear_grad(*[b2.gated_linear(x, w)[0], x, w, b2.gated_linear(x, w, want_z=True)[1]])

    def step():
        h, z = b2.gated_linear(x, w, want_z=True)
        return (h, z) + b2.gated_linear_grad(h, x, w, z)
    torch.cuda.synchronize()
    graphs, outs = [torch.cuda.CUDAGraph() for _ in range(2)], []
    for one in graphs:
        with torch.cuda.graph(one):
            outs.append(step())
    for seed in (1, 2):
        x.copy_(tensor(gen(seed), (50, 131), torch.float16))
        for one in graphs:
            one.replay()
        want = step()
        for out in outs:
            assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_another_stream_and_given_outputs():
    g = gen(13)
    x, w = tensor(g, (70, 256), torch.bfloat16), tensor(g, (192, 256), torch.bfloat16, 0.1)
    want = b2.gated_linear(x, w, want_z=True)
    grads = b2.gated_linear_grad(want[0], x, w, want[1])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    h, z = torch.empty_like(want[0]), torch.empty_like(want[1])
    got = b2.gated_linear(x, w, h=h, z=z, stream=st)
    gg = b2.gated_linear_grad(want[0], x, w, want[1], stream=st)
    torch.cuda.current_stream().wait_stream(st)
    assert got[0] is h and got[1] is z
    assert torch.equal(h, want[0]) and torch.equal(z, want[1])
    assert all(torch.equal(a, b) for a, b in zip(gg, grads))


def test_results_past_2_31_elements():
    """z of more than 2^31 elements: its last rows against the same rows by themselves."""
    rows, n_in, n_out = (1 << 31) // 16384 + 300, 64, 8192
    g = gen(14)
    x = tensor(g, (rows, n_in), torch.bfloat16)
    w = tensor(g, (2 * n_out, n_in), torch.bfloat16, 0.1)
    h, z = b2.gated_linear(x, w, want_z=True)
    last, lz = b2.gated_linear(x[-300:].contiguous(), w, want_z=True)
    dx, _, _ = b2.gated_linear_grad(h, x, w, z, want_weight=False, want_bias=False)
    d, _, _ = b2.gated_linear_grad(last, x[-300:].contiguous(), w, lz, want_weight=False,
                                   want_bias=False)
    # other tilings, so other orders of the sums: a last place (2^-7 at most, relative) turned
    # here and there; wrong rows would be off by their whole size
    for a, b in ((h[-300:], last), (z[-300:], lz), (dx[-300:], d)):
        assert float((a.float() - b.float()).norm() / b.float().norm()) <= 2.0 ** -8


# -- float32 products in pieces: rows, in, out with 9 rows and 2^26 products or more -----------

PIECES = [(700, 640, 160), (513, 1027, 131), (20, 2048, 1700), (40, 1500, 1200), (2100, 128, 260),
          (90, 520, 1537), (10, 4096, 3300),
          (5, 4095, 3300)]


@pytest.mark.parametrize("rows,n_in,n_out", PIECES)
def test_float32_in_pieces(rows, n_in, n_out):
    """Within the bounds of binary32 sums, and in the norm better than a binary32 step; the
    gradients too."""
    check_forward(rows, n_in, n_out, torch.float32, seed=21)
    g = gen(22)
    x, w = tensor(g, (rows, n_in), torch.float32), tensor(g, (2 * n_out, n_in), torch.float32, 0.05)
    dh = tensor(g, (rows, n_out), torch.float32, 0.3)
    z = tensor(g, (rows, 2 * n_out), torch.float32)
    ref, bound = G.gated_grad(dh.cpu(), x.cpu(), w.cpu(), z.cpu(), "silu")
    got = b2.gated_linear_grad(dh, x, w, z)
    for a, r, e, name in zip(got, ref, bound, ("dx", "dw", "db")):
        assert_within(a, r, e, name)
        assert float((a.double().cpu() - r).norm() / r.norm()) <= 8 * 2.0 ** -24, name
    for i, one in enumerate((dict(want_weight=False, want_bias=False),
                             dict(want_input=False, want_bias=False),
                             dict(want_input=False, want_weight=False))):
        assert torch.equal(b2.gated_linear_grad(dh, x, w, z, **one)[i], got[i])


@pytest.mark.parametrize("tiling", TILINGS)
def test_every_tiling_in_pieces(tiling):
    """Whole numbers with 11 and 13 bits, which need two pieces each; sums stay below 2^24 (2^35
    by magnitude in pieces' products, each exact), so that every bit is known."""
    rows, n_in, n_out = (16, 2112, 2001) if tiling[3] else (300, 640, 363)
    assert b2.library().b200norm_testing_force_linear(*tiling) == 0
    g = gen(23)
    x = torch.randint(-1500, 1501, (rows, n_in), generator=g, device="cuda")
    x *= torch.rand(x.shape, generator=g, device="cuda") < 0.01
    w = torch.randint(-400, 401, (2 * n_out, n_in), generator=g, device="cuda")
    want = x.double() @ w.double().t()
    assert float((x.double().abs() @ w.double().abs().t()).max()) < 2 ** 24
    h, z = b2.gated_linear(x.float(), w.float(), activation=0, want_z=True)
    assert torch.equal(z.double(), want)
    assert torch.equal(h, (want[:, :n_out].float() * want[:, n_out:].float()))


@pytest.mark.parametrize("rows,n_in,n_out,tiling", [
    (64, 448, 2400, (0, 0, 0, 0)), (64, 448, 2400, (1, 64, 8, 1)), (30, 384, 6000, (1, 32, 8, 1)),
    (64, 320, 3300, (1, 64, 8, 1)), (16, 192, 22000, (1, 16, 8, 1)), (300, 448, 520, (1, 128, 8, 0)),
    (700, 150, 700, (1, 128, 8, 0))])
def test_more_parts_than_slices_in_pieces(rows, n_in, n_out, tiling):
    """A part of a sum may have no slice of 64 (448 are seven, in eight parts): in whole numbers,
    exactly; and an infinity of another part is not lost."""
    assert b2.library().b200norm_testing_force_linear(*tiling) == 0
    g = gen(33)
    x = torch.randint(-1500, 1501, (rows, n_in), generator=g, device="cuda")
    x *= torch.rand(x.shape, generator=g, device="cuda") < 0.05
    w = torch.randint(-300, 301, (2 * n_out, n_in), generator=g, device="cuda")
    want = x.double() @ w.double().t()
    assert float((x.double().abs() @ w.double().abs().t()).max()) < 2 ** 24
    h, z = b2.gated_linear(x.float(), w.float(), activation=0, want_z=True)
    assert torch.equal(z.double(), want)
    assert torch.equal(h, (want[:, :n_out].float() * want[:, n_out:].float()))
    bad = x.float()
    bad[rows - 1, n_in - 1] = float("inf")
    z = b2.gated_linear(bad, w.float(), activation=0, want_z=True)[1]
    assert torch.equal(z[:-1].double(), want[:-1])
    same_specials(z[-1:], product(bad[-1:], w.float()), "row")


def test_the_gradients_tilings_in_pieces():
    """The same of both products of a gradient: z of gates 1 without an activation, so that dz
    is dh twice."""
    rows, n_in, n_out = 333, 580, 420
    g = gen(24)
    x = torch.randint(-300, 301, (rows, n_in), generator=g, device="cuda")
    w = torch.randint(-300, 301, (2 * n_out, n_in), generator=g, device="cuda")
    dh = torch.randint(-700, 701, (rows, n_out), generator=g, device="cuda")
    dh *= torch.rand(dh.shape, generator=g, device="cuda") < 0.05
    z = torch.ones(rows, 2 * n_out, device="cuda")
    dz = torch.cat((dh, dh), 1).double()
    wants = dz @ w.double(), dz.t() @ x.double(), dz.sum(0)
    assert max(float((dz.abs() @ w.double().abs()).max()),
               float((dz.abs().t() @ x.double().abs()).max())) < 2 ** 24
    for tiling in [(0, 0, 0, 0), (2, 256, 1, 0), (1, 128, 1, 0), (1, 128, 4, 0), (1, 64, 1, 0),
                   (1, 64, 8, 0)]:
        assert b2.library().b200norm_testing_force_linear(*tiling) == 0
        got = b2.gated_linear_grad(dh.float(), x.float(), w.float(), z, activation=0)
        for a, want in zip(got, wants):
            assert torch.equal(a.double(), want), tiling


def test_pieces_of_any_magnitude():
    """Rows from 2^-60 to 2^60 in size, and a row of the largest numbers: each is as accurate as
    the others.  What is not finite stays in its row or column."""
    rows, n_in, n_out = 121, 1024, 600
    g = gen(25)
    x = tensor(g, (rows, n_in), torch.float32)
    x *= (2.0 ** torch.arange(-60, 61, device="cuda")).unsqueeze(1)
    w = tensor(g, (2 * n_out, n_in), torch.float32, 0.03)
    _, z = b2.gated_linear(x, w, want_z=True)
    want = x.double() @ w.double().t()
    off = (z.double() - want).norm(dim=1) / want.norm(dim=1)
    assert float(off.max()) <= 8 * 2.0 ** -24
    top = torch.finfo(torch.float32).max
    big = torch.zeros_like(x)
    big[:, 0] = top
    small = torch.full_like(w, 2.0 ** -130)
    _, z = b2.gated_linear(big, small, want_z=True)
    # The tensor cores cut a sum at 2^-24 or less of the largest product of its operands'
    # exponents, and a subnormal operand's counts as 2^-126: 2^-24 * 2^(128 - 126) each time, and
    # here one addition mixes numbers (the other pieces' products are alone in theirs).
    assert float(z.sub(top * 2.0 ** -130).abs().max()) <= 2.0 ** -24 * 2.0 ** 2
    bad = x.clone()
    bad[5, 7], bad[9, 1] = float("nan"), float("inf")
    h, _ = b2.gated_linear(bad, w)
    keep = torch.ones(rows, dtype=torch.bool, device="cuda")
    keep[5] = keep[9] = False
    assert torch.equal(h[keep], b2.gated_linear(x, w)[0][keep])
    assert bool(torch.isnan(h[5]).all()) and not bool(torch.isfinite(h[9]).any())


def kind(v):
    """0 finite, 1 and -1 the infinities, 2 NaN."""
    return torch.where(torch.isnan(v), 2, torch.isposinf(v).int() - torch.isneginf(v).int())


def same_specials(got, wants, name):
    """NaN, infinities and finite values where one of the references has them.  There are two for
    a product of finite values past binary32 that meets an infinity of the other sign: -inf +
    3.9998e38 is -inf where one multiply-add makes it, and NaN where the sum is split, as the part
    with 3.9998e38 > 2^128 (1 - 2^-25) alone has the sum +inf."""
    ok = torch.zeros_like(got, dtype=torch.bool)
    for want in wants:
        ok |= kind(got) == kind(want.float())
    assert bool(ok.all()), (name, (~ok).nonzero()[:5])


def product(a, b):
    """a b^T in binary64, term by term: the terms as they are, and rounded to binary32."""
    return [torch.stack([f(r, b).double().sum(-1) for r in a])
            for f in (lambda r, b: r.double() * b.double(), lambda r, b: r * b)]


@pytest.mark.parametrize("tiling", [(0, 0, 0, 0)] + TILINGS)
def test_infinities_and_overflow_in_pieces(tiling):
    """What is not finite is what binary32 products of the values give, whatever their pieces'
    products do: pieces that are zero, pieces of the other sign, first and second pieces whose
    product overflows alone.  No other sum is another."""
    rows, n_in, n_out = (16, 2112, 2001) if tiling[3] else (300, 640, 363)
    assert b2.library().b200norm_testing_force_linear(*tiling) == 0
    g = gen(27)
    x, w = tensor(g, (rows, n_in), torch.float32), tensor(g, (2 * n_out, n_in), torch.float32)
    inf, last = float("inf"), rows - 1
    w[:, 3] = torch.where(w[:, 3] > 0, 1.0, -1.0)      # one piece, the others zero
    w[5, 3] = w[n_out + 7, 3] = 0.0                     # infinity times zero
    clean = b2.gated_linear(x, w, activation=0, want_z=True)
    assert all(bool(torch.isfinite(v).all()) for v in clean)
    bad = x.clone()
    bad[0, 3] = inf
    bad[2, 100] = -inf
    bad[4, 3], bad[4, n_in - 1] = inf, inf              # infinities of both signs meet
    bad[6, 8] = torch.finfo(torch.float32).max          # overflows with most weights
    bad[8, 9] = -1.99609375 * 2.0 ** 127                # its pieces: -2^128 + 2^119, cut
    bad[last, 3], bad[last, 5] = inf, float("nan")
    wide = w.clone()
    wide[:, 8] *= 2.0 ** 20
    wide[:, 9] = torch.where(wide[:, 9] > 0, 1.0, -1.0) * (1 + 2.0 ** -9) * 2.0 ** 2
    want = product(bad[[0, 2, 4, 6, 8, last]], wide)
    z = b2.gated_linear(bad, wide, activation=0, want_z=True)[1]
    same_specials(z[[0, 2, 4, 6, 8, last]], want, "rows")
    assert bool(torch.isinf(want[0].float()[[0, 1, 3, 4]]).any(1).all())
    keep = torch.ones(rows, dtype=torch.bool, device="cuda")
    keep[[0, 2, 4, 6, 8, last]] = False
    assert torch.equal(z[keep], b2.gated_linear(x, wide, activation=0, want_z=True)[1][keep])
    # the same in the weight: a gate's feature, one of what it gates, and the last ones
    bad = w.clone()
    features = [1, n_out - 1, n_out, 2 * n_out - 1, n_out + 9, 12]
    bad[1, 3], bad[n_out - 1, 7], bad[n_out, 7] = inf, -inf, inf
    bad[2 * n_out - 1, n_in - 1] = inf
    bad[n_out + 9, 4], bad[12, 4] = (s * torch.finfo(torch.float32).max for s in (1, -1))
    wide = x.clone()
    wide[:, 4] *= 8.0
    h, z = b2.gated_linear(wide, bad, activation=0, want_z=True)
    same_specials(z[:, features], [v.t() for v in product(bad[features], wide)], "features")
    keep = torch.ones(2 * n_out, dtype=torch.bool, device="cuda")
    keep[features] = False
    base = b2.gated_linear(wide, w, activation=0, want_z=True)[1]
    assert torch.equal(z[:, keep], base[:, keep])
    same_specials(h, [z[:, :n_out] * z[:, n_out:]], "h")


@pytest.mark.parametrize("tiling", [(0, 0, 0, 0), (2, 256, 1, 0), (1, 128, 1, 0), (1, 128, 4, 0),
                                    (1, 64, 1, 0), (1, 64, 8, 0)])
def test_infinities_and_overflow_of_gradients_in_pieces(tiling):
    """The same of dx and dw."""
    rows, n_in, n_out = 333, 580, 420
    assert b2.library().b200norm_testing_force_linear(*tiling) == 0
    g = gen(28)
    x, w = tensor(g, (rows, n_in), torch.float32), tensor(g, (2 * n_out, n_in), torch.float32)
    dh, z = tensor(g, (rows, n_out), torch.float32), tensor(g, (rows, 2 * n_out), torch.float32)
    inf = float("inf")
    z[rows - 1, 11], z[rows - 1, n_out + 11] = 1.0, 0.0
    clean = b2.gated_linear_grad(dh, x, w, z, activation=0)
    bad = dh.clone()
    bad[0, 2], bad[40, n_out - 1], bad[rows - 1, 11] = inf, -inf, 2.0 ** 127
    xb, wb = x.clone(), w.clone()
    xb[7, 20], xb[9, n_in - 1] = inf, float("nan")
    wb[3, 30], wb[n_out + 5, 0] = -inf, inf
    dx, dw, _ = b2.gated_linear_grad(bad, xb, wb, z, activation=0)
    dz = torch.cat((bad * z[:, n_out:], bad * z[:, :n_out]), 1)
    rx, rw = [0, 40, rows - 1, 1, 2, 200], [2, n_out + 2, n_out - 1, 11, n_out + 11, 50]
    same_specials(dx[rx], product(dz[rx], wb.t()), "dx")
    same_specials(dw[rw], product(dz.t()[rw], xb.t()), "dw")
    cols = torch.ones(n_in, dtype=torch.bool, device="cuda")
    cols[[30, 0]] = False
    assert torch.equal(dx[1:40][:, cols], clean[0][1:40][:, cols])
    cols[:] = True
    cols[[20, n_in - 1]] = False
    one = [i for i in range(2 * n_out) if i % n_out not in (2, 11, n_out - 1)]
    assert torch.equal(dw[one][:, cols], clean[1][one][:, cols])


def test_nothing_finite_in_pieces():
    """Every sum made again: the waits allow for it, and the results are as above."""
    rows, n_in, n_out = 600, 1024, 512
    g = gen(29)
    w = tensor(g, (2 * n_out, n_in), torch.float32).abs() + 0.1
    for value in (float("nan"), float("inf"), -float("inf")):
        x = torch.full((rows, n_in), value, device="cuda")
        h, z = b2.gated_linear(x, w, activation=0, want_z=True)
        b2.linear_status()
        same_specials(z, [torch.full_like(z, value)], "z")
        dx, dw, _ = b2.gated_linear_grad(x[:, :n_out].contiguous(), x, w, torch.ones_like(z),
                                         activation=0)
        b2.linear_status()
        assert not bool(torch.isfinite(dx).any()) and not bool(torch.isfinite(dw).any())


@pytest.mark.parametrize("tiling", [(2, 256, 1, 0), (1, 128, 1, 0), (1, 128, 4, 0), (1, 16, 2, 1)])
def test_waits_in_pieces_give_up(tiling):
    lib = b2.library()
    g = gen(26)
    x, w = tensor(g, (16, 2048), torch.float32), tensor(g, (2 * 2200, 2048), torch.float32)
    assert lib.b200norm_testing_force_linear(*tiling) == 0
    want, _ = b2.gated_linear(x, w)
    b2.linear_status()
    try:
        for stall in (True, False):
            if stall:
                assert lib.b200norm_testing_linear_stall(1, 20_000_000) == 0
            else:
                assert lib.b200norm_testing_linear_withhold(1, 20_000_000) == 0
            t0 = time.monotonic()
            b2.gated_linear(x, w)
            with pytest.raises(b2.B200NormError) as e:
                b2.linear_status()
            assert e.value.status == TIMEOUT and time.monotonic() - t0 < 5.0
            assert lib.b200norm_testing_linear_stall(0, 0) == 0
    finally:
        lib.b200norm_testing_linear_withhold(0, 0)
    b2.linear_status()
    assert torch.equal(b2.gated_linear(x, w)[0], want)

"""GPU: rotation and RMS norm of query and key heads against binary64."""
import math

import pytest
import torch

import head_formulas as H
import residual_add_normalization_gb300 as b2
from formulas import DTYPES, assert_within

pytestmark = pytest.mark.gpu

EPS = 1e-6


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def frequencies(rot, base=10000.0):
    return base ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / max(rot, 1))


def heads(g, shape, t, how, extra=1):
    """Heads (batch, seq, n, size) that lie in memory as `how` says, and their storage."""
    b, s, n, d = shape
    if how == "rows":        # inside a product's rows, between other heads
        base = torch.randn(b, s, n + 2 * extra, d, generator=g, device="cuda").to(t)
        return base[:, :, extra:extra + n], base
    if how == "permuted":    # head by head
        base = torch.randn(b, n, s, d, generator=g, device="cuda").to(t)
        return base.transpose(1, 2), base
    if how == "odd":         # at no 16-byte boundary
        base = torch.randn(b * s * n * d + 1, generator=g, device="cuda").to(t)
        return base[1:].view(b, s, n, d), base
    base = torch.randn(b, s, n, d, generator=g, device="cuda").to(t)
    return base, base


SIZES = [(1, 0), (2, 2), (7, 6), (16, 16), (33, 4), (40, 20), (64, 64), (64, 16), (80, 40),
         (80, 80), (96, 96), (128, 128), (128, 64), (128, 6), (130, 130), (192, 64), (256, 256),
         (320, 80), (512, 512), (576, 64), (1000, 1000), (1023, 2), (1024, 1024), (128, 0)]


def both(q, k, positions, freq, interleaved, scale, t, m, seed, gamma=True):
    """Forward of both forms and the gradients, of q and k together, against binary64."""
    g = gen(seed)
    size = q.shape[-1]
    gq, gk = ((torch.randn(size, generator=g, device="cuda") * 0.2 + 1).to(m) for _ in range(2))
    if not gamma:
        gk = None
    turn = H.turn_of(positions.cpu(), freq.cpu(), scale)
    for inverse in (False, True):
        got = b2.rotary(q, k, positions, freq, interleaved=interleaved, scale=scale,
                        inverse=inverse)
        for v, x, name in zip(got, (q, k), "qk"):
            ref, bound = H.rotary(x.cpu(), turn.conj() if inverse else turn, interleaved)
            assert_within(v, ref, bound, f"rotary {name} inverse={inverse}")
    got = b2.head_rms_rotary(q, k, gq, gk, positions, freq, epsilon=EPS, interleaved=interleaved,
                             scale=scale)
    for v, x, w, name in zip(got, (q, k), (gq, gk), "qk"):
        ref, bound = H.head_norm(x.cpu(), None if w is None else w.cpu(), turn, EPS, interleaved)
        assert_within(v, ref, bound, f"norm {name}")
    dq, dk = ((torch.randn(v.shape, generator=g, device="cuda") * 0.3).to(t) for v in (q, k))
    dxq, dxk, dgq, dgk = b2.head_rms_rotary_grad(dq, dk, q, k, gq, gk, positions, freq,
                                                 epsilon=EPS, interleaved=interleaved, scale=scale)
    for dx, dg, d, x, w, name in ((dxq, dgq, dq, q, gq, "q"), (dxk, dgk, dk, k, gk, "k")):
        (rx, rg), (ex, eg) = H.head_norm_grad(d.cpu(), x.cpu(), None if w is None else w.cpu(),
                                              turn, EPS, interleaved)
        assert_within(dx, rx, ex, f"dx of {name}")
        assert (dg is None) == (w is None)
        if dg is not None:
            assert_within(dg, rg, eg, f"dgamma of {name}")


@pytest.mark.parametrize("t", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("size,rot", SIZES)
def test_sizes(size, rot, interleaved, t):
    g = gen(size * 7 + rot)
    q, _ = heads(g, (2, 5, 6, size), DTYPES[t], "rows")
    k, _ = heads(g, (2, 5, 3, size), DTYPES[t], "dense")
    positions = torch.randint(0, 5000, (2, 5), generator=g, device="cuda")
    both(q, k, positions, frequencies(rot), interleaved, 1.0, DTYPES[t], DTYPES[t], 1)


@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("size,rot", [
    (9, 8), (17, 10), (20, 20), (36, 20), (50, 26), (96, 24), (98, 98), (100, 52), (100, 100),
    (129, 64), (130, 66), (150, 150), (252, 252), (254, 6), (257, 256), (260, 100), (300, 300),
    (508, 508), (510, 510), (512, 508), (516, 516)])
def test_rows_in_few_lanes(size, rot, interleaved, t):
    """Accesses of 2, 4 and 8 bytes, with one unit of a lane to sixteen, rows that fill their
    lanes and rows that do not."""
    g = gen(size * 11 + rot)
    q, _ = heads(g, (1, 7, 5, size), DTYPES[t], "rows")
    k, _ = heads(g, (1, 7, 3, size), DTYPES[t], "dense")
    positions = torch.randint(0, 5000, (1, 7), generator=g, device="cuda")
    both(q, k, positions, frequencies(rot), interleaved, 1.0, DTYPES[t], torch.float32, 1)


@pytest.mark.parametrize("t,m", [("bf16", "f32"), ("f16", "f16"), ("f32", "f32")])
@pytest.mark.parametrize("how", ["dense", "rows", "permuted", "odd"])
@pytest.mark.parametrize("batch,seq,nq,nk", [(1, 1, 1, 1), (1, 1, 32, 8), (3, 1, 33, 1),
                                             (1, 257, 4, 4), (5, 63, 7, 2), (2, 1500, 3, 1)])
def test_layouts(batch, seq, nq, nk, how, t, m):
    g = gen(batch * 100 + seq)
    q, _ = heads(g, (batch, seq, nq, 64), DTYPES[t], how)
    k, _ = heads(g, (batch, seq, nk, 64), DTYPES[t], how)
    start = torch.randint(-100, 100000, (batch, 1), generator=g, device="cuda")
    positions = (start + torch.arange(seq, device="cuda")).int()
    both(q, k, positions, frequencies(32, 500000.0), seq % 2 == 0, 1.25, DTYPES[t], DTYPES[m], 2,
         gamma=batch != 3)


@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("nq,nk", [(1, 1), (1, 0), (0, 1), (6, 1), (1, 6)])
@pytest.mark.parametrize("size,step", [(128, 129), (64, 67), (40, 41), (36, 37), (34, 35),
                                       (256, 1 << 61)])
def test_one_head_with_any_step(size, step, nq, nk, t):
    """The step between the heads of a tensor that has one is not taken: it may be odd where the
    tokens are whole vectors apart, or reach past any memory.  The lanes without a row must not
    go by it either."""
    g = gen(size + nq)

    def one(n):
        if n == 0:
            return None
        if n > 1:
            return torch.randn(2, 9, n, size, generator=g, device="cuda").to(DTYPES[t])
        base = torch.randn(2 * 9 * 8 * 136 + 256, generator=g, device="cuda").to(DTYPES[t])
        return base.as_strided((2, 9, 1, size), (9 * 1032, 1032, step, 1))
    q, k, dq, dk = one(nq), one(nk), one(nq), one(nk)
    p, f = torch.randint(0, 5000, (2, 9), generator=g, device="cuda"), frequencies(size)
    gamma = torch.randn(size, generator=g, device="cuda")
    gq, gk = gamma if nq else None, gamma if nk else None

    def run(q, k, dq, dk):
        return (b2.rotary(q, k, p, f) + b2.head_rms_rotary(q, k, gq, gk, p, f)
                + b2.head_rms_rotary_grad(dq, dk, q, k, gq, gk, p, f))
    same = [None if v is None else v.contiguous().clone() for v in (q, k, dq, dk)]
    for got, want in zip(run(q, k, dq, dk), run(*same)):
        assert (got is None and want is None) or torch.equal(got, want)
    if nq and nk:
        both(q, k, p, f, False, 1.0, DTYPES[t], torch.float32, 3)


@pytest.mark.parametrize("t", ["bf16", "f32"])
def test_positions_by_sequence_or_for_all(t):
    """(seq,) positions serve every sequence, a column that steps over others as well."""
    g = gen(3)
    q, _ = heads(g, (3, 10, 4, 32), DTYPES[t], "dense")
    table = torch.randint(0, 1 << 20, (10, 7), generator=g, device="cuda")
    one = table[:, 2]
    f = frequencies(32)
    want = b2.rotary(q, None, one.expand(3, 10).contiguous(), f)[0]
    assert torch.equal(b2.rotary(q, None, one, f)[0], want)
    assert torch.equal(b2.rotary(q, None, one.expand(3, 10), f)[0], want)
    assert torch.equal(b2.rotary(None, q, one.int(), f)[1], want)
    flat = b2.rotary(q.view(30, 4, 32), None, one.repeat(3), f)[0]
    assert torch.equal(flat.view(3, 10, 4, 32), want)


@pytest.mark.parametrize("first", [(1 << 31) - 2, (1 << 40) - 3, -(1 << 35), (1 << 62), -(1 << 63)])
def test_far_positions(first):
    """Frequencies of whole 2^-20 turns: the angle is known exactly at any position, up to
    the 2^-53 of p f that the frequency's own rounding allows (2^-54 for it, 2^-54 for the
    quotient); from 2^45 on nothing but whole turns is asked for."""
    turns = torch.tensor([1, 1 << 10, 1 << 19], dtype=torch.float64)
    freq = (turns * 2 * math.pi / (1 << 20)).cuda()
    p = torch.tensor([first, first + 1], dtype=torch.int64)
    # p * turns mod 2^20, in whole numbers
    exact = torch.tensor([[(int(v) * int(n)) % (1 << 20) for n in turns] for v in p],
                         dtype=torch.float64) / (1 << 20) * 2 * math.pi
    slack = p.double().abs().unsqueeze(-1) * turns * 2 * math.pi / (1 << 20) * 2.0 ** -51
    x = torch.zeros(2, 1, 6, device="cuda")
    x[..., :3] = 1.0
    y = b2.rotary(x, None, p.cuda(), freq)[0].cpu().double()[:, 0]
    ok = ((y[:, :3] - exact.cos()).abs() <= slack + H.ROT + 2.0 ** -24) | (slack > 0.1)
    ok &= ((y[:, 3:] - exact.sin()).abs() <= slack + H.ROT + 2.0 ** -24) | (slack > 0.1)
    assert bool(ok.all())
    assert bool((y[:, :3] ** 2 + y[:, 3:] ** 2 - 1).abs().max() <= 20 * H.ROT)


@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_frequencies_that_are_not_finite(t, interleaved):
    """Their pairs are NaN, at position 0 as well; no other element is another, and the gradient's
    rows are NaN where they have such a pair."""
    g = gen(15)
    x, _ = heads(g, (1, 6, 3, 40), DTYPES[t], "dense")
    p = torch.tensor([[0, 1, -1, 7, 100000, 1 << 40]], device="cuda")
    f = frequencies(32)
    # half a turn, and a step of binary64 more: the numbers next to what stands for no angle
    f[4], f[5] = math.pi, math.pi + 2.0 ** -51
    bad = f.clone()
    where = {1: float("nan"), 3: float("inf"), 9: -float("inf")}
    for i, v in where.items():
        bad[i] = v
    spoilt = torch.zeros(40, dtype=torch.bool, device="cuda")
    for i in where:
        spoilt[[2 * i, 2 * i + 1] if interleaved else [i, i + 16]] = True
    for inverse in (False, True):
        y = b2.rotary(x, None, p, bad, interleaved=interleaved, inverse=inverse)[0]
        want = b2.rotary(x, None, p, f, interleaved=interleaved, inverse=inverse)[0]
        assert bool(torch.isfinite(want).all())
        assert bool(torch.isnan(y[..., spoilt]).all())
        assert torch.equal(y[..., ~spoilt], want[..., ~spoilt])
    y = b2.head_rms_rotary(x, None, None, None, p, bad, interleaved=interleaved)[0]
    want = b2.head_rms_rotary(x, None, None, None, p, f, interleaved=interleaved)[0]
    assert bool(torch.isnan(y[..., spoilt]).all())
    assert torch.equal(y[..., ~spoilt], want[..., ~spoilt])
    gamma = torch.ones(40, device="cuda")
    dx, _, dg, _ = b2.head_rms_rotary_grad(x, None, x, None, gamma, None, p, bad,
                                           interleaved=interleaved)
    assert bool(torch.isnan(dx).all())
    assert torch.equal(torch.isnan(dg), spoilt)


def test_every_angle():
    """Cosine and sine of 2^20 angles over a turn, and of the smallest ones."""
    n = 1 << 20
    x = torch.zeros(n, 1, 2, device="cuda")
    x[..., 0] = 1.0
    for freq in (2 * math.pi / n, 1e-9):
        p = torch.arange(n, device="cuda")
        y = b2.rotary(x, None, p, torch.tensor([freq], dtype=torch.float64, device="cuda"))[0]
        angle = p.double() * freq
        off = (y[:, 0].double() - torch.stack((angle.cos(), angle.sin()), -1)).abs().max()
        assert float(off) <= 9 * 2.0 ** -24 + 2.0 ** -25


@pytest.mark.parametrize("t", ["bf16", "f32"])
def test_a_token_alone_gives_the_batch_s_bits(t):
    g = gen(5)
    q, _ = heads(g, (2, 300, 32, 128), DTYPES[t], "rows")
    k, _ = heads(g, (2, 300, 8, 128), DTYPES[t], "rows")
    gq, gk = (torch.randn(128, generator=g, device="cuda").to(DTYPES[t]) for _ in range(2))
    p = torch.arange(600, device="cuda").view(2, 300)
    f = frequencies(128)
    yq, yk = b2.head_rms_rotary(q, k, gq, gk, p, f)
    for b, s in ((0, 0), (1, 299), (0, 77)):
        aq, ak = b2.head_rms_rotary(q[b, s:s + 1], k[b, s:s + 1], gq, gk, p[b, s:s + 1], f)
        assert torch.equal(aq[0], yq[b, s]) and torch.equal(ak[0], yk[b, s])
    assert torch.equal(b2.head_rms_rotary(q, None, gq, None, p, f)[0], yq)
    assert torch.equal(b2.head_rms_rotary(None, k, None, gk, p, f)[1], yk)


@pytest.mark.parametrize("size,rot,t", [(128, 128, "bf16"), (80, 40, "f16"), (33, 32, "f32")])
def test_in_place_and_into_rows(size, rot, t):
    """In place, and into views of one tensor: the bits of the plain call, and nothing else
    is touched."""
    g = gen(6)
    base = torch.randn(3, 50, 11, size, generator=g, device="cuda").to(DTYPES[t])
    q, k = base[:, :, 1:7], base[:, :, 7:9]
    p, f = torch.arange(50, device="cuda"), frequencies(rot)
    gamma = torch.randn(size, generator=g, device="cuda")
    want = b2.head_rms_rotary(q, k, gamma, gamma, p, f)
    into = torch.full_like(base, 7.0)
    out = b2.head_rms_rotary(q, k, gamma, gamma, p, f, q_out=into[:, :, 2:8],
                             k_out=into[:, :, 8:10])
    assert out[0].data_ptr() == into[:, :, 2:8].data_ptr()
    for v, w in zip(out, want):
        assert torch.equal(v, w)
    assert bool((into[:, :, :2] == 7).all()) and bool((into[:, :, 10:] == 7).all())
    keep = base.clone()
    b2.head_rms_rotary(q, k, gamma, gamma, p, f, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(base[:, :, :1], keep[:, :, :1])
    assert torch.equal(base[:, :, 9:], keep[:, :, 9:])
    # permuted results
    dst = torch.full((3, 6, 51, size), 7.0, device="cuda").to(DTYPES[t])
    view = dst[:, :, :50].transpose(1, 2)
    b2.rotary(keep[:, :, 1:7], None, p, f, q_out=view)
    assert torch.equal(view, b2.rotary(keep[:, :, 1:7], None, p, f)[0])
    assert bool((dst[:, :, 50] == 7).all())


@pytest.mark.parametrize("shape", [(2, 9, 4, 3, 64), (1, 9, 4, 3, 64), (2, 1, 4, 3, 64),
                                   (2, 9, 1, 3, 64), (9, 2, 5, 3, 20)])
@pytest.mark.parametrize("order", [(0, 1, 2, 3), (2, 0, 1, 3), (0, 3, 1, 2), (3, 2, 1, 0)])
def test_queries_keys_and_values_side_by_side_in_any_axis(shape, order):
    """In place and into views of one tensor, where queries, keys and values alternate head by
    head, or the axes lie in another order: the bits of dense results, and values as they were.
    `order`: the axes (batch, seq, head, which of the three) from the outermost."""
    g = gen(16)
    lie = torch.randn([shape[i] for i in order] + [shape[4]], generator=g, device="cuda").bfloat16()
    view = lie.permute([order.index(i) for i in range(4)] + [4])
    q, k, v = view.unbind(3)
    p, f = torch.arange(shape[1], device="cuda"), frequencies(shape[4])
    gamma = torch.randn(shape[4], generator=g, device="cuda")
    want = b2.head_rms_rotary(q, k, gamma, gamma, p, f)
    dq, dk = (torch.randn(w.shape, generator=g, device="cuda").bfloat16() for w in want)
    grads = b2.head_rms_rotary_grad(dq, dk, q, k, gamma, gamma, p, f)
    into = torch.full_like(lie, 7.0)
    gq, gk, gv = into.permute([order.index(i) for i in range(4)] + [4]).unbind(3)
    got = b2.head_rms_rotary_grad(dq, dk, q, k, gamma, gamma, p, f, dq_out=gq, dk_out=gk)
    assert all(torch.equal(a, b) for a, b in zip(got, grads)) and bool((gv == 7).all())
    keep = v.clone()
    b2.head_rms_rotary(q, k, gamma, gamma, p, f, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(v, keep)


@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_nan_and_infinity_stay_where_they_are(t, interleaved):
    """A NaN row spoils no other row, elements that are not rotated keep their bits, and an
    infinity reaches its own pair only."""
    g = gen(8)
    x, _ = heads(g, (1, 9, 5, 96), DTYPES[t], "dense")
    p, f = torch.arange(9, device="cuda"), frequencies(44)
    clean = b2.rotary(x, None, p, f, interleaved=interleaved)[0]
    norm = b2.head_rms_rotary(x, None, None, None, p, f, interleaved=interleaved)[0]
    bad = x.clone()
    bad[0, 4, 2, 10] = float("inf")
    bad[0, 4, 2, 60] = float("nan")
    y = b2.rotary(bad, None, p, f, interleaved=interleaved)[0]
    pair = (10, 11) if interleaved else (10, 32)
    same = torch.ones(96, dtype=torch.bool)
    same[list(pair)] = False
    same[60] = False
    assert torch.equal(y[0, 4, 2][same.cuda()], clean[0, 4, 2][same.cuda()])
    assert bool(torch.isnan(y[0, 4, 2, 60]))
    assert not bool(torch.isfinite(y[0, 4, 2, list(pair)]).any())
    yn = b2.head_rms_rotary(bad, None, None, None, p, f, interleaved=interleaved)[0]
    rows = torch.ones(9, 5, dtype=torch.bool, device="cuda")
    rows[4, 2] = False
    assert torch.equal(y[0][rows], clean[0][rows]) and torch.equal(yn[0][rows], norm[0][rows])
    assert bool(torch.isnan(yn[0, 4, 2]).all())
    dx = b2.head_rms_rotary_grad(x, None, bad, None, None, None, p, f, interleaved=interleaved)[0]
    ok = b2.head_rms_rotary_grad(x, None, x, None, None, None, p, f, interleaved=interleaved)[0]
    assert torch.equal(dx[0][rows], ok[0][rows])


@pytest.mark.parametrize("size,lanes", [(24, 1), (128, 8)])
def test_zero_rows_without_epsilon(size, lanes):
    """0 / 0 is NaN by the definition, in its own row; other rows' sums are not spoiled by
    lanes that hold no row."""
    x = torch.ones(1, 5, size, device="cuda")
    dy = torch.ones_like(x)
    _, _, dg, _ = b2.head_rms_rotary_grad(dy, None, x, None, torch.ones(size, device="cuda"), None,
                                          None, None, epsilon=0.0)
    assert torch.equal(dg, torch.full((size,), 5.0, device="cuda"))
    x[0, 3] = 0
    y = b2.head_rms_rotary(x, None, None, None, None, None, epsilon=0.0)[0]
    assert bool(torch.isnan(y[0, 3]).all())
    assert torch.equal(y[0, :3], torch.ones(3, size, device="cuda"))


@pytest.mark.parametrize("t", ["bf16", "f16", "f32"])
def test_gradient_of_many_rows(t):
    """Enough tokens that every part takes several; shared gammas' sums are exact in whole
    numbers: u = +-1, da = whole numbers without a rotation."""
    rows, n, d = 3001, 12, 64
    g = gen(9)
    sign = torch.randint(0, 2, (rows, n, d), generator=g, device="cuda") * 2 - 1
    dy = torch.randint(-3, 4, (rows, n, d), generator=g, device="cuda")
    gamma = torch.ones(d, device="cuda")
    out = b2.head_rms_rotary_grad(dy.to(DTYPES[t]), dy[:, :5].to(DTYPES[t]), sign.to(DTYPES[t]),
                                  sign[:, :5].to(DTYPES[t]), gamma, gamma, None, None, epsilon=0.0)
    assert torch.equal(out[2].double(), (dy * sign).sum((0, 1)).double())
    assert torch.equal(out[3].double(), (dy * sign)[:, :5].sum((0, 1)).double())
    again = b2.head_rms_rotary_grad(dy.to(DTYPES[t]), dy[:, :5].to(DTYPES[t]),
                                    sign.to(DTYPES[t]), sign[:, :5].to(DTYPES[t]), gamma, gamma,
                                    None, None, epsilon=0.0)
    for a, b in zip(out, again):
        assert torch.equal(a, b)


def test_gradient_against_differences():
    """dx and dgamma of float32 heads against central differences of the binary64 formula."""
    g = gen(10)
    x, dy = (torch.randn(2, 3, 10, generator=g, device="cuda") for _ in range(2))
    gamma = torch.randn(10, generator=g, device="cuda")
    p = torch.tensor([3, 70], device="cuda")
    f = frequencies(8)
    dx, _, dg, _ = b2.head_rms_rotary_grad(dy, None, x, None, gamma, None, p, f, scale=1.5)
    turn = H.turn_of(p.cpu(), f.cpu(), 1.5)
    xd, gd, dyd = x.cpu().double(), gamma.cpu().double(), dy.cpu().double()

    def loss(xv, gv):
        return float((H.head_norm(xv, gv, turn, 1e-6, False)[0] * dyd).sum())
    h = 1e-5
    for at in [(0, 0, 0), (1, 2, 9), (0, 1, 5), (1, 0, 3)]:
        e = torch.zeros_like(xd)
        e[at] = h
        want = (loss(xd + e, gd) - loss(xd - e, gd)) / (2 * h)
        assert abs(float(dx[at]) - want) <= 1e-5 * (1 + abs(want))
    for at in range(10):
        e = torch.zeros_like(gd)
        e[at] = h
        want = (loss(xd, gd + e) - loss(xd, gd - e)) / (2 * h)
        assert abs(float(dg[at]) - want) <= 1e-5 * (1 + abs(want))


def test_nothing_wanted_and_nothing_there():
    x = torch.ones(4, 2, 8, device="cuda")
    gamma = torch.ones(8, device="cuda")
    p, f = torch.arange(4, device="cuda"), frequencies(8)
    assert b2.head_rms_rotary_grad(x, x, x, x, gamma, gamma, p, f, want_input=False,
                                   want_gamma=False) == (None, None, None, None)
    dx, _, dg, dgk = b2.head_rms_rotary_grad(x, x, x, x, gamma, gamma, p, f, want_input=False)
    assert dx is None and dg is not None and dgk is not None
    dx, dk, dg, _ = b2.head_rms_rotary_grad(x, x, x, x, gamma, gamma, p, f, want_gamma=False)
    assert dg is None and dx is not None and dk is not None
    for shape in ((0, 2, 8), (2, 0, 2, 8), (3, 4, 0, 8)):
        e = torch.ones(shape, device="cuda")
        pe = torch.zeros(shape[:-2], dtype=torch.int64, device="cuda")
        assert b2.rotary(e, None, pe, f)[0].shape == e.shape
        y = b2.head_rms_rotary(e, e, gamma, gamma, pe, f)
        assert y[0].shape == e.shape
        if shape[-2]:
            dx, _, dg, _ = b2.head_rms_rotary_grad(e, None, e, None, gamma, None, pe, f)
            assert dx.shape == e.shape and bool((dg == 0).all())


@pytest.mark.parametrize("m", ["bf16", "f32"])
@pytest.mark.parametrize("nq,nk", [(0, 0), (0, 3), (3, 0)])
@pytest.mark.parametrize("tokens", [(5,), (2, 5), (0,)])
def test_gammas_without_heads_have_gradients_of_zeros(tokens, nq, nk, m):
    """Given and new ones, beside those of a tensor that has heads and by themselves."""
    g = gen(14)
    q, k = (torch.randn(*tokens, n, 8, generator=g, device="cuda").bfloat16() for n in (nq, nk))
    gamma = torch.rand(8, generator=g, device="cuda").to(DTYPES[m])
    p, f = torch.zeros(tokens, dtype=torch.int64, device="cuda"), frequencies(8)
    want = [torch.zeros_like(gamma) if v.numel() == 0 else
            b2.head_rms_rotary_grad(v, None, v, None, gamma, None, p, f)[2] for v in (q, k)]
    for _ in range(3):  # in memory that has been used
        torch.full((1 << 16,), float("nan"), device="cuda")
        out = b2.head_rms_rotary_grad(q, k, q, k, gamma, gamma, p, f)
        assert torch.equal(out[2], want[0]) and torch.equal(out[3], want[1])
        assert out[0].shape == q.shape and out[1].shape == k.shape
    into = [torch.full_like(gamma, 7.0) for _ in range(2)]
    out = b2.head_rms_rotary_grad(q, k, q, k, gamma, gamma, p, f, want_input=False,
                                  dgamma_q=into[0], dgamma_k=into[1])
    assert out[2] is into[0] and torch.equal(into[0], want[0]) and torch.equal(into[1], want[1])
    alone = b2.head_rms_rotary_grad(q, None, q, None, gamma, None, p, f)[2]
    assert torch.equal(alone, want[0])


def test_offsets_past_32_bits():
    """Tokens more than 2^31 elements apart."""
    step = (1 << 31) + 8
    base = torch.zeros(step + 4096, dtype=torch.bfloat16, device="cuda")
    x = base.as_strided((2, 3, 128), (step, 128, 1))
    x.copy_(torch.randn(2, 3, 128, generator=gen(11), device="cuda"))
    p, f = torch.tensor([5, 9], device="cuda"), frequencies(128)
    want = b2.rotary(x.contiguous(), None, p, f)[0]
    assert torch.equal(b2.rotary(x, None, p, f)[0], want)
    out = torch.zeros(step + 4096, dtype=torch.bfloat16, device="cuda").as_strided(
        (2, 3, 128), (step, 128, 1))
    b2.rotary(x, None, p, f, q_out=out)
    assert torch.equal(out, want)
    g = b2.head_rms_rotary_grad(x, None, x, None, None, None, p, f)[0]
    c = x.contiguous()
    assert torch.equal(g, b2.head_rms_rotary_grad(c, None, c, None, None, None, p, f)[0])


def test_captured_and_replayed():
    """A graph takes new positions and heads at each replay, gradients with their workspace
    among them, while other calls run in between."""
    g = gen(12)
    q, k = (torch.randn(4, n, 64, generator=g, device="cuda").bfloat16() for n in (8, 2))
    gamma = torch.randn(64, generator=g, device="cuda")
    p, f = torch.arange(4, device="cuda"), frequencies(64)

    def both_ways():
        y = b2.head_rms_rotary(q, k, gamma, gamma, p, f)
        return y + b2.head_rms_rotary_grad(y[0], y[1], q, k, gamma, gamma, p, f)
    both_ways()
    torch.cuda.synchronize()
    graph, second = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both_ways()
    with torch.cuda.graph(second):
        out2 = both_ways()
    for seed in (1, 2):
        h = gen(seed)
        q.copy_(torch.randn(4, 8, 64, generator=h, device="cuda"))
        p.copy_(torch.randint(0, 1 << 20, (4,), generator=h, device="cuda"))
        graph.replay()
        second.replay()
        want = both_ways()
        for a, b, c in zip(out, out2, want):
            assert torch.equal(a, c) and torch.equal(b, c)


def test_another_stream():
    g = gen(13)
    q = torch.randn(700, 16, 128, generator=g, device="cuda").bfloat16()
    gamma = torch.ones(128, device="cuda")
    p, f = torch.arange(700, device="cuda"), frequencies(128)
    want = b2.head_rms_rotary(q, None, gamma, None, p, f)[0]
    wg = b2.head_rms_rotary_grad(q, None, q, None, gamma, None, p, f)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = b2.head_rms_rotary(q, None, gamma, None, p, f, stream=st)[0]
    gg = b2.head_rms_rotary_grad(q, None, q, None, gamma, None, p, f, stream=st)
    torch.cuda.current_stream().wait_stream(st)
    assert torch.equal(got, want) and torch.equal(gg[0], wg[0]) and torch.equal(gg[2], wg[2])

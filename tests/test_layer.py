"""GPU: layer normalization and its gradients against binary64 formulas, at the
sizes, types and values where they can go wrong."""
import math

import pytest
import torch

import formulas as F
import residual_add_normalization_gb300 as b2

pytestmark = pytest.mark.gpu



@pytest.fixture(autouse=True)
def _no_wait_gave_up():
    yield
    b2.rows_status()


EPS = 1e-5
TYPES = [("f32", "f32"), ("f16", "f16"), ("f16", "f32"), ("bf16", "bf16"), ("bf16", "f32")]
# rows x hidden: one element, less than a vector, odd widths, every schedule's
# range, rows of one and more rows than CTAs
SHAPES = [(1, 1), (3, 5), (2, 8), (5, 33), (64, 64), (7, 100), (65, 768), (33, 1027), (3, 4096),
          (700, 1024), (2, 8200), (3, 20000), (2, 70001)]


def make(rows, hidden, t, m, seed, offset=0.5):
    g = torch.Generator().manual_seed(seed)

    def n(shape, dt, scale=1.0, mean=0.0):
        return (torch.randn(shape, generator=g) * scale + mean).to(F.DTYPES[dt])
    return dict(x=n((rows, hidden), t, 1.0, offset), skip=n((rows, hidden), t),
                bias=n((hidden,), t, 0.1), gamma=n((hidden,), m, 0.1, 1.0),
                beta=n((hidden,), m, 0.1), dy=n((rows, hidden), t, 0.3),
                ds=n((rows, hidden), t, 0.3))


def dev(v, shift=0):
    """On the GPU; with `shift`, starting that many elements into its block."""
    if v is None:
        return None
    if not shift:
        return v.cuda()
    flat = torch.empty(v.numel() + shift, dtype=v.dtype, device="cuda")
    out = flat[shift:].view(v.shape)
    out.copy_(v)
    return out


def check_forward(d, t, skip, bias, beta, shift=0):
    sk, bi, be = (d["skip"] if skip else None, d["bias"] if bias else None,
                  d["beta"] if beta else None)
    y, s, mean, inv = b2.skip_layer_stats(
        dev(d["x"], shift), dev(sk, shift), dev(d["gamma"], shift), dev(be, shift),
        dev(bi, shift), epsilon=EPS)
    rs = F.residual_sum(d["x"], sk, bi)
    assert torch.equal(s.cpu(), rs)
    ry, rmean, rinv, bound = F.layer(rs, d["gamma"], be, EPS)
    F.assert_within(y, ry, bound, "y")
    n = rs.shape[-1]
    depth = 8 * math.ceil(n / 4096) + n % 8 + 16
    F.assert_within(mean, rmean, depth * F.U * rs.double().abs().mean(-1, keepdim=True), "mean")
    dm = depth * F.U * rs.double().abs().mean(-1, keepdim=True)
    F.assert_within(inv, rinv, rinv * ((depth + 6) * F.U + (rinv * dm) ** 2), "inv_std_var")


@pytest.mark.parametrize("t,m", TYPES)
@pytest.mark.parametrize("rows,hidden", SHAPES)
def test_forward(rows, hidden, t, m):
    d = make(rows, hidden, t, m, rows * 31 + hidden)
    check_forward(d, t, True, True, True)
    check_forward(d, t, False, False, hidden % 2 == 0)


@pytest.mark.parametrize("t,m", TYPES)
@pytest.mark.parametrize("rows,hidden", [(9, 64), (17, 1024), (3, 4096), (2, 20000)])
def test_forward_unaligned(rows, hidden, t, m):
    check_forward(make(rows, hidden, t, m, hidden), t, True, True, True, shift=1)


@pytest.mark.parametrize("rows,hidden", [(5, 96), (9, 1024), (4, 4096), (3, 70000)])
def test_forward_offset_costs_no_digits(rows, hidden):
    """A common offset a thousand times the spread: the centred squares keep
    their digits (a difference of mean squares would lose six)."""
    check_forward(make(rows, hidden, "f32", "f32", hidden, offset=1000.0), "f32", False, False,
                  True)


def test_forward_same_without_outputs():
    """y does not depend on which other outputs are asked for."""
    d = {k: dev(v) for k, v in make(40, 4096, "bf16", "bf16", 1).items()}
    a = (d["x"], d["skip"], d["gamma"], d["beta"], d["bias"])
    y0, s0, _, _ = b2.skip_layer_stats(*a, epsilon=EPS)
    y1, s1 = b2.skip_layer(*a, epsilon=EPS, want_sum=False)
    assert s1 is None and torch.equal(y0, y1)
    y2, s2 = b2.skip_layer(s0, None, d["gamma"], d["beta"], epsilon=EPS)
    assert s2 is s0 and torch.equal(y0, y2)


def test_forward_special_values():
    """A constant row gives beta; a NaN or an infinity stays in its row."""
    x = torch.randn(6, 1024)
    x[1] = 3.0
    x[2, 5] = math.nan
    x[4, 1000] = math.inf
    g, b = torch.rand(1024) + 0.5, torch.randn(1024)
    y, _, mean, inv = b2.skip_layer_stats(x.cuda(), None, g.cuda(), b.cuda(), epsilon=EPS)
    y = y.cpu()
    assert torch.equal(y[1], b)
    assert y[2].isnan().all() and y[4].isnan().all()
    for r in (0, 3, 5):
        ry, _, _, bound = F.layer(x[r:r + 1], g, b, EPS)
        F.assert_within(y[r:r + 1], ry, bound, "y")


def check_grad(d, ds, bias, shift=0):
    s = d["x"]
    _, mean, inv, _ = F.layer(s, d["gamma"], None, EPS)
    mean, inv = mean.float(), inv.float()
    dsv = d["ds"] if ds else None
    got = b2.skip_layer_grad(dev(d["dy"], shift), dev(s, shift), dev(mean), dev(inv),
                             dev(d["gamma"], shift), ds=dev(dsv, shift), want_bias=bias)
    ref, bound = F.layer_grad(d["dy"], s, mean, inv, d["gamma"], dsv)
    for name, g, r, b in zip(("dx", "dgamma", "dbeta", "dbias"), got, ref, bound):
        if name == "dbias" and not bias:
            assert g is None
            continue
        F.assert_within(g, r, b, name)
    return got


@pytest.mark.parametrize("t,m", TYPES)
@pytest.mark.parametrize("rows,hidden", SHAPES + [(3000, 40), (1300, 4096)])
def test_grad(rows, hidden, t, m):
    d = make(rows, hidden, t, m, rows * 17 + hidden)
    check_grad(d, True, True)
    check_grad(d, False, False)


@pytest.mark.parametrize("t,m", TYPES)
@pytest.mark.parametrize("rows,hidden", [(9, 64), (170, 1024), (3, 4096), (2, 20000)])
def test_grad_unaligned(rows, hidden, t, m):
    check_grad(make(rows, hidden, t, m, hidden), True, True, shift=1)


# Many rows that are not whole 16-byte vectors: one row or more per CTA, rows of one
# to several CTAs, every shift, a last row whose last vector is cut
ODD_SHAPES = [(40001, 67), (20400, 131), (3000, 1027), (1300, 2050), (700, 4095), (330, 8195),
              (141, 20001), (61, 50003)]


@pytest.mark.parametrize("t,m", TYPES)
@pytest.mark.parametrize("rows,hidden", ODD_SHAPES)
def test_forward_many_odd_rows(rows, hidden, t, m):
    d = make(rows, hidden, t, m, rows + hidden)
    check_forward(d, t, True, True, True)
    check_forward(d, t, False, False, False)


@pytest.mark.parametrize("t,m", TYPES)
@pytest.mark.parametrize("rows,hidden", ODD_SHAPES + [(6100, 129), (800, 1027), (13, 65001)])
def test_grad_many_odd_rows(rows, hidden, t, m):
    d = make(rows, hidden, t, m, rows + hidden)
    check_grad(d, True, True)
    check_grad(d, False, False)


@pytest.mark.parametrize("t,m", TYPES)
@pytest.mark.parametrize("rows,hidden", [(400, 9000), (300, 16384), (130, 32768), (50, 65536)])
def test_grad_many_long_rows(rows, hidden, t, m):
    """More rows than clusters of CTAs, of two to eight CTAs each."""
    d = make(rows, hidden, t, m, rows + hidden)
    check_grad(d, True, True)
    check_grad(d, False, False)


@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("rows,hidden", [(3000, 1027), (330, 8195)])
def test_many_odd_rows_special_values(rows, hidden, t):
    """NaN and infinities stay in their rows, whose elements share vectors with
    those of their neighbours, and in dgamma and dbeta in their columns."""
    d = make(rows, hidden, t, t, 12)
    clean = {k: dev(v) for k, v in d.items()}
    bad = {k: v.clone() for k, v in clean.items()}
    marked = [1, 8, rows // 2, rows - 1]
    for i, r in enumerate(marked):
        bad["x"][r, 0 if i % 2 else hidden - 1] = math.nan if i < 2 else math.inf
    keep = torch.ones(rows, dtype=torch.bool, device="cuda")
    keep[marked] = False
    args = ("skip", "gamma", "beta", "bias")
    want = b2.skip_layer_stats(clean["x"], *(clean[k] for k in args), epsilon=EPS)
    got = b2.skip_layer_stats(bad["x"], *(bad[k] for k in args), epsilon=EPS)
    for w, g in zip(want, got):
        assert torch.equal(w[keep], g[keep])
    assert bool(torch.isnan(got[0][~keep].float()).all())
    bad["dy"][marked, 5] = math.nan
    stats = want[1:]
    dx, dg, db, dc = b2.skip_layer_grad(clean["dy"], *stats, clean["gamma"], want_bias=True)
    bx, bg, bb, bc = b2.skip_layer_grad(bad["dy"], *stats, bad["gamma"], want_bias=True)
    assert torch.equal(dx[keep], bx[keep]) and bool(torch.isnan(bx[~keep].float()).all())
    for w, g in ((dg, bg), (db, bb)):
        columns = torch.isnan(g.float())
        assert bool(columns[5]) and int(columns.sum()) == 1
        assert torch.equal(w[~columns], g[~columns])
    assert bool(torch.isnan(bc.float()).all())


def test_grad_wanted_outputs():
    """Each output alone has the bits it has among the others; equal calls give
    equal bits."""
    d = make(500, 768, "bf16", "f32", 3)
    whole = check_grad(d, True, True)
    _, mean, inv, _ = F.layer(d["x"], d["gamma"], None, EPS)
    a = [v.cuda() for v in (d["dy"], d["x"], mean.float(), inv.float(), d["gamma"])]
    ds = d["ds"].cuda()
    off = dict(want_input=False, want_gamma=False, want_beta=False, want_bias=False)
    for i, w in enumerate(off):
        got = b2.skip_layer_grad(*a, ds=ds, **{**off, w: True})
        assert [g is None for g in got] == [j != i for j in range(4)]
        assert torch.equal(got[i], whole[i]), w


@pytest.mark.parametrize("t,m", [("f32", "f32"), ("bf16", "bf16")])
def test_grad_no_rows(t, m):
    x = torch.empty(0, 64, dtype=F.DTYPES[t], device="cuda")
    e = torch.empty(0, 1, device="cuda")
    g = torch.ones(64, dtype=F.DTYPES[m], device="cuda")
    dx, dg, db, dc = b2.skip_layer_grad(x, x, e, e, g, want_bias=True)
    assert dx.shape == (0, 64)
    assert not dg.any() and not db.any() and not dc.any()
    y, s = b2.skip_layer(x, None, g)
    assert y.shape == (0, 64)


@pytest.mark.parametrize("rows,hidden", [(4, 48), (3, 1024)])
def test_grad_against_differences(rows, hidden):
    """The loss sum(dy * y) along a random direction in (S, gamma, beta):
    central differences of the binary64 forward against the kernel's gradients."""
    d = make(rows, hidden, "f32", "f32", 5)
    x, g, b, dy = (d[k].double() for k in ("x", "gamma", "beta", "dy"))
    gen = torch.Generator().manual_seed(6)
    vx, vg, vb = (torch.randn(v.shape, generator=gen, dtype=torch.float64) for v in (x, g, b))

    def loss(h):
        return (dy * F.layer(x + h * vx, g + h * vg, b + h * vb, EPS)[0]).sum()
    h = 1e-5
    want = (loss(h) - loss(-h)) / (2 * h)
    y, s, mean, inv = b2.skip_layer_stats(d["x"].cuda(), None, d["gamma"].cuda(),
                                          d["beta"].cuda(), epsilon=EPS)
    dx, dg, db, _ = (None if v is None else v.cpu().double() for v in b2.skip_layer_grad(
        d["dy"].cuda(), s, mean, inv, d["gamma"].cuda()))
    got = (dx * vx).sum() + (dg * vg).sum() + (db * vb).sum()
    scale = (dx * vx).abs().sum() + (dg * vg).abs().sum() + (db * vb).abs().sum()
    # differences: third-order term h^2 and cancellation 1e-16 / h; kernel: U per term
    assert abs(got - want) <= 1e-6 * scale


def test_on_a_stream_of_its_own_and_in_a_graph():
    d = {k: dev(v) for k, v in make(300, 4096, "f16", "f16", 8).items()}
    a = (d["x"], d["skip"], d["gamma"], d["beta"], d["bias"])
    y0, s0, mean0, inv0 = b2.skip_layer_stats(*a, epsilon=EPS)
    g0 = b2.skip_layer_grad(d["dy"], s0, mean0, inv0, d["gamma"], ds=d["ds"], want_bias=True)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    y1, s1, mean1, inv1 = b2.skip_layer_stats(*a, epsilon=EPS, stream=st)
    g1 = b2.skip_layer_grad(d["dy"], s1, mean1, inv1, d["gamma"], ds=d["ds"], want_bias=True,
                            stream=st)
    st.synchronize()
    assert torch.equal(y0, y1) and all(torch.equal(p, q) for p, q in zip(g0, g1))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y2, s2, mean2, inv2 = b2.skip_layer_stats(*a, epsilon=EPS)
        g2 = b2.skip_layer_grad(d["dy"], s2, mean2, inv2, d["gamma"], ds=d["ds"], want_bias=True)
    d["x"].add_(1.0)
    graph.replay()
    y3, s3, mean3, inv3 = b2.skip_layer_stats(*a, epsilon=EPS)
    g3 = b2.skip_layer_grad(d["dy"], s3, mean3, inv3, d["gamma"], ds=d["ds"], want_bias=True)
    torch.cuda.synchronize()
    assert torch.equal(y2, y3) and all(torch.equal(p, q) for p, q in zip(g2, g3))


@pytest.mark.parametrize("rows,hidden,shift", [(5, 4096, 0), (37, 64, 0), (7, 1027, 1),
                                               (600, 768, 0), (3001, 1027, 0),
                                               (331, 8195, 0)])
def test_writes_exactly_its_outputs(rows, hidden, shift):
    """Outputs inside 0xFF-filled blocks: nothing beside them changes, and the
    workspace's size is enough."""
    d = {k: dev(v) for k, v in make(rows, hidden, "bf16", "f32", hidden).items()}

    def guarded(shape, dtype):
        es = torch.finfo(dtype).bits // 8
        n = math.prod(shape) * es
        raw = torch.full((4096 + shift * es + n + 4096,), 0xFF, dtype=torch.uint8, device="cuda")
        a = 4096 + shift * es
        return raw, raw[a:a + n].view(dtype).view(shape), a, n
    t, m = torch.bfloat16, torch.float32
    blocks = [guarded(s, k) for s, k in (((rows, hidden), t), ((rows, hidden), t),
                                         ((rows, hidden), t), ((hidden,), m), ((hidden,), m),
                                         ((hidden,), t))]
    o = [b[1] for b in blocks]
    _, _, mean, inv = b2.skip_layer_stats(d["x"], d["skip"], d["gamma"], d["beta"], d["bias"],
                                          output=o[0], sum_out=o[1])
    need = b2.library().b200norm_skip_layer_grad_workspace_size(rows, hidden)
    ws = torch.full((need + 4096,), 0xFF, dtype=torch.uint8, device="cuda")
    b2.skip_layer_grad(d["dy"], o[1], mean, inv, d["gamma"], dx=o[2], dgamma=o[3], dbeta=o[4],
                       dbias=o[5], workspace=ws[:need])
    torch.cuda.synchronize()
    assert bool((ws[need:] == 0xFF).all())
    for raw, view, a, n in blocks:
        assert bool((raw[:a] == 0xFF).all()) and bool((raw[a + n:] == 0xFF).all())
        assert not bool(torch.isnan(view.float()).any())


def test_threads_on_one_stream():
    """Several threads' gradient calls on one stream: each has its own scratch, so
    their launches may interleave."""
    import threading
    cases = [{k: dev(v) for k, v in make(200, 1024, "bf16", "f32", 30 + i).items()}
             for i in range(4)]
    stats = [b2.skip_layer_stats(d["x"], None, d["gamma"])[2:] for d in cases]

    def call(i):
        return b2.skip_layer_grad(cases[i]["dy"], cases[i]["x"], *stats[i], cases[i]["gamma"])[:3]
    want = [call(i) for i in range(4)]
    torch.cuda.synchronize()
    wrong, errors = [], []

    def work(i):
        try:
            for _ in range(50):
                if not all(torch.equal(g, w) for g, w in zip(call(i), want[i])):
                    wrong.append(i)
        except Exception as e:  # noqa: BLE001
            errors.append(e)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors and not wrong

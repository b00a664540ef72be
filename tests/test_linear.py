"""GPU: the linear operator and its gradients against binary64 formulas, at the
sizes, types and values where they can go wrong."""
import math

import pytest
import torch

import formulas as F
import residual_add_normalization_gb300 as b2

pytestmark = pytest.mark.gpu

ACTS = ["none", "silu", "gelu", "gelu_tanh", "relu"]
# rows x in x out: single elements and tokens, sizes around every tile edge,
# rows that are not whole 16-byte vectors, long sums
SHAPES = [(1, 1, 1), (1, 64, 64), (1, 4096, 520), (2, 16, 24), (3, 5, 7), (5, 72, 130),
          (8, 1000, 129), (16, 512, 256), (17, 264, 264), (33, 65, 1000), (64, 768, 768),
          (65, 64, 72), (127, 128, 136), (128, 128, 128), (129, 136, 256), (130, 1027, 99),
          (200, 2048, 320), (256, 320, 512), (257, 520, 264), (300, 8200, 64), (513, 72, 1283),
          (2, 4096, 1030), (3, 2051, 1030), (4, 1030, 1500)]


@pytest.fixture(autouse=True)
def _no_wait_gave_up():
    yield
    b2.library().b200norm_testing_force_linear(0, 0, 0, 0)
    b2.linear_status()


def make(rows, n_in, n_out, t, seed):
    g = torch.Generator().manual_seed(seed)

    def n(shape, scale=1.0):
        return (torch.randn(shape, generator=g) * scale).to(F.DTYPES[t])
    return dict(x=n((rows, n_in)), w=n((n_out, n_in), 1.5 / math.sqrt(n_in)),
                bias=n((n_out,), 0.5), residual=n((rows, n_out)), dy=n((rows, n_out), 0.3),
                z=n((rows, n_out), 1.5))


def dev(v, shift=0):
    if v is None:
        return None
    if not shift:
        return v.cuda()
    flat = torch.empty(v.numel() + shift, dtype=v.dtype, device="cuda")
    out = flat[shift:].view(v.shape)
    out.copy_(v)
    return out


def check_forward(d, name, bias, residual, keep, shift=0):
    bi, re = d["bias"] if bias else None, d["residual"] if residual else None
    y, z = b2.linear(dev(d["x"], shift), dev(d["w"], shift), dev(bi, shift), dev(re, shift),
                     activation=F.ACTIVATIONS[name], want_z=keep)
    (ry, rz), (ey, ez) = F.linear(d["x"], d["w"], bi, re, name)
    F.assert_within(y, ry, ey, "y")
    if ry.numel() > 64:
        F.assert_rms(y, ry, y.dtype, d["x"].shape[-1], "y")
    if keep:
        F.assert_within(z, rz, ez, "z")
    else:
        assert z is None
    return y


@pytest.mark.parametrize("t", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward(shape, t):
    d = make(*shape, t, sum(shape))
    check_forward(d, "none", True, True, False)
    check_forward(d, ACTS[1 + sum(shape) % 4], sum(shape) % 3 > 0, False, True)


@pytest.mark.parametrize("t", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("shape", [(3, 64, 40), (130, 64, 300)])
def test_forward_activations(shape, name, t):
    check_forward(make(*shape, t, 5), name, True, True, True)


@pytest.mark.parametrize("t", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("shape", [(1, 256, 64), (7, 1027, 33), (130, 136, 264)])
def test_forward_unaligned(shape, t):
    check_forward(make(*shape, t, 9), "gelu", True, True, True, shift=1)


@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 200])
def test_forward_special_values(rows, t):
    """A NaN or an infinity stays in its row of x and its column of weight."""
    d = make(rows, 96, 72, t, 4)
    d["x"][0, 3] = math.inf
    d["w"][5, 7] = math.nan
    y, _ = b2.linear(d["x"].cuda(), d["w"].cuda())
    ref = d["x"].double() @ d["w"].double().t()
    y = y.cpu().double()
    assert torch.equal(y.isnan(), ref.isnan()) and torch.equal(y.isinf(), ref.isinf())
    assert y[:, 5].isnan().all() and not y[1:, :5].isnan().any()


def test_forward_rows_do_not_depend_on_z():
    d = make(96, 512, 384, "bf16", 2)
    a = [d[k].cuda() for k in ("x", "w", "bias", "residual")]
    y0, _ = b2.linear(*a, activation=2)
    y1, z1 = b2.linear(*a, activation=2, want_z=True)
    assert torch.equal(y0, y1)


def check_grad(d, name, shift=0):
    z = d["z"] if name != "none" else None
    got = b2.linear_grad(dev(d["dy"], shift), dev(d["x"], shift), dev(d["w"], shift),
                         dev(z, shift), activation=F.ACTIVATIONS[name])
    ref, bound = F.linear_grad(d["dy"], d["x"], d["w"], z, name)
    rows, n_out = d["dy"].shape
    for what, g, r, e, terms in zip(("dx", "dw", "db"), got, ref, bound, (n_out, rows, rows)):
        F.assert_within(g, r, e, what)
        if r.numel() > 64 and r.norm() > 0:
            F.assert_rms(g, r, g.dtype, terms, what)
    return got


@pytest.mark.parametrize("t", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("shape", SHAPES)
def test_grad(shape, t):
    d = make(*shape, t, sum(shape) + 1)
    check_grad(d, "none")
    check_grad(d, ACTS[1 + sum(shape) % 4])


@pytest.mark.parametrize("t", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("name", ACTS)
def test_grad_activations(name, t):
    d = make(70, 64, 136, t, 6)
    d["z"][0, :8] = torch.tensor([0.0, -0.0, 20.0, -20.0, 200.0, -200.0, 5.5, -5.5])
    check_grad(d, name)


@pytest.mark.parametrize("name", ["silu", "gelu", "gelu_tanh", "relu"])
def test_grad_infinite_z(name):
    """act' is 0 or 1 far out, also at the infinities."""
    d = make(4, 8, 8, "f32", 6)
    d["z"][0, :4] = torch.tensor([math.inf, -math.inf, 3e38, -3e38])
    _, _, db = b2.linear_grad(*(d[k].cuda() for k in ("dy", "x", "w", "z")),
                              activation=F.ACTIVATIONS[name])
    z = d["z"].clone()
    z[0, :4] = torch.tensor([300.0, -300.0, 300.0, -300.0])
    ref, bound = F.linear_grad(d["dy"], d["x"], d["w"], z, name)
    F.assert_within(db, ref[2], bound[2], "db")


@pytest.mark.parametrize("t", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("shape", [(1, 256, 64), (70, 1027, 33), (130, 136, 264)])
def test_grad_unaligned(shape, t):
    check_grad(make(*shape, t, 9), "silu", shift=1)
    check_grad(make(*shape, t, 9), "none", shift=1)


@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("name", ["none", "gelu"])
def test_grad_wanted_outputs(name, t):
    d = make(150, 136, 264, t, 3)
    whole = check_grad(d, name)
    z = d["z"].cuda() if name != "none" else None
    a = [d[k].cuda() for k in ("dy", "x", "w")] + [z]
    off = dict(want_input=False, want_weight=False, want_bias=False)
    for i, w in enumerate(off):
        got = b2.linear_grad(*a, activation=F.ACTIVATIONS[name], **{**off, w: True})
        assert [g is None for g in got] == [j != i for j in range(3)]
        assert torch.equal(got[i], whole[i]), w


@pytest.mark.parametrize("t", ["bf16", "f32"])
def test_no_rows(t):
    x = torch.empty(0, 64, dtype=F.DTYPES[t], device="cuda")
    w = torch.ones(32, 64, dtype=F.DTYPES[t], device="cuda")
    y, _ = b2.linear(x, w)
    assert y.shape == (0, 32)
    dx, dw, db = b2.linear_grad(y, x, w)
    assert dx.shape == (0, 64) and not dw.any() and not db.any()


@pytest.mark.parametrize("name", ACTS)
def test_grad_against_differences(name):
    """The loss sum(dy * y) along a random direction in (x, w, b): central
    differences of the binary64 forward against the kernels' gradients."""
    d = make(24, 40, 56, "f32", 7)
    x, w, b, dy = (d[k].double() for k in ("x", "w", "bias", "dy"))
    gen = torch.Generator().manual_seed(8)
    vx, vw, vb = (torch.randn(v.shape, generator=gen, dtype=torch.float64) for v in (x, w, b))

    def loss(h):
        return (dy * F.linear(x + h * vx, w + h * vw, b + h * vb, None, name)[0][0]).sum()
    h = 1e-6
    want = (loss(h) - loss(-h)) / (2 * h)
    _, z = b2.linear(d["x"].cuda(), d["w"].cuda(), d["bias"].cuda(),
                     activation=F.ACTIVATIONS[name], want_z=True)
    got = [v.cpu().double() for v in b2.linear_grad(d["dy"].cuda(), d["x"].cuda(), d["w"].cuda(),
                                                    z, activation=F.ACTIVATIONS[name])]
    parts = [(g * v) for g, v in zip(got, (vx, vw, vb))]
    scale = sum(p.abs().sum() for p in parts)
    # a kink of ReLU within h of a z is as likely as h; its share of the loss is h as well
    assert abs(sum(p.sum() for p in parts) - want) <= 2e-6 * scale


@pytest.mark.parametrize("t", ["bf16", "f32"])
def test_on_a_stream_of_its_own_and_in_a_graph(t):
    d = {k: v.cuda() for k, v in make(160, 1027, 272, t, 8).items()}

    def both(**kw):
        y, z = b2.linear(d["x"], d["w"], d["bias"], d["residual"], activation=2, want_z=True, **kw)
        return (y, z) + b2.linear_grad(d["dy"], d["x"], d["w"], z, activation=2, **kw)
    first = both()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    second = both(stream=st)
    st.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(first, second))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        third = both()
    d["x"].add_(0.5)
    graph.replay()
    fourth = both()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(third, fourth))


@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("shape,shift", [((5, 64, 40), 0), ((130, 136, 264), 0), ((70, 99, 33), 1),
                                         ((1, 512, 256), 0), ((300, 256, 512), 0)])
def test_writes_exactly_its_outputs(shape, shift, t):
    rows, n_in, n_out = shape
    d = {k: dev(v, shift) for k, v in make(*shape, t, 1).items()}
    dt = F.DTYPES[t]
    es = torch.finfo(dt).bits // 8

    def guarded(s):
        n = math.prod(s) * es
        raw = torch.full((4096 + shift * es + n + 4096,), 0xFF, dtype=torch.uint8, device="cuda")
        a = 4096 + shift * es
        return raw, raw[a:a + n].view(dt).view(s), a, n
    blocks = [guarded(s) for s in ((rows, n_out), (rows, n_out), (rows, n_in), (n_out, n_in),
                                   (n_out,))]
    o = [b[1] for b in blocks]
    lib, code = b2.library(), {"f32": 0, "f16": 1, "bf16": 2}[t]
    need = (lib.b200norm_linear_workspace_size(rows, n_in, n_out, code, 0 if shift else 1),
            lib.b200norm_linear_grad_workspace_size(rows, n_in, n_out, code, 1,
                                                    0 if shift else 1))
    ws = [torch.full((n + 4096,), 0xFF, dtype=torch.uint8, device="cuda") for n in need]
    b2.linear(d["x"], d["w"], d["bias"], d["residual"], activation=1, y=o[0], z=o[1],
              workspace=ws[0][:need[0]])
    b2.linear_grad(d["dy"], d["x"], d["w"], o[1], activation=1, dx=o[2], dw=o[3], db=o[4],
                   workspace=ws[1][:need[1]])
    torch.cuda.synchronize()
    for w, n in zip(ws, need):
        assert bool((w[n:] == 0xFF).all())
    for raw, view, a, n in blocks:
        assert bool((raw[:a] == 0xFF).all()) and bool((raw[a + n:] == 0xFF).all())
        assert not bool(torch.isnan(view.float()).any())


TILINGS = [(2, 256, 1), (1, 128, 1), (1, 128, 2), (1, 128, 8), (1, 64, 1), (1, 64, 4), (1, 64, 8)]


@pytest.mark.parametrize("t", ["bf16", "f16"])
@pytest.mark.parametrize("tiling", TILINGS)
@pytest.mark.parametrize("shape", [(1, 512, 8), (300, 520, 264), (520, 1032, 784),
                                   (257, 4104, 129)])
def test_every_tiling(shape, tiling, t):
    """The tilings that the sizes of the other tests may not take, at sizes with
    ragged edges; (520, 1032, 784) has more tiles than one."""
    d = make(*shape, t, 11)
    assert b2.library().b200norm_testing_force_linear(*tiling, 0) == 0
    check_forward(d, "silu", True, True, True)
    if shape[0] >= 512 and shape[2] % 8 == 0:  # long enough sums of every product
        check_grad(d, "gelu_tanh")


@pytest.mark.parametrize("t", ["bf16", "f16"])
@pytest.mark.parametrize("bn,splits", [(16, 1), (16, 8), (32, 2), (32, 8), (64, 1), (64, 4)])
@pytest.mark.parametrize("rows", [1, 16])
def test_every_tiling_for_few_rows(rows, bn, splits, t):
    d = make(rows, 776, 1000, t, 12)
    assert b2.library().b200norm_testing_force_linear(1, bn, splits, 1) == 0
    check_forward(d, "gelu", True, True, True)


@pytest.mark.parametrize("shape", [(20, 4096, 24), (40, 2000, 130), (17, 300, 64), (9, 1030, 7)])
def test_float32_sums_in_parts(shape):
    """Few tiles and long sums: K split over clusters, and the last part ragged."""
    d = make(*shape, "f32", 14)
    check_forward(d, "gelu", True, True, True)
    check_grad(d, "silu")


@pytest.mark.parametrize("tiling", [(2, 256), (1, 128), (1, 64)])
@pytest.mark.parametrize("keep,residual", [(False, False), (False, True), (True, False)])
def test_more_tiles_than_ctas(tiling, keep, residual):
    """Several tiles per CTA: the buffers of sums and of results in turn, also
    past the last column's edge (a 64-column piece of a tile is left out)."""
    d = make(2600, 136, 4360, "bf16", 13)
    assert b2.library().b200norm_testing_force_linear(*tiling, 1, 0) == 0
    for _ in range(3):
        check_forward(d, "none", True, residual, keep)


def test_threads_on_one_stream():
    """Several threads' gradient calls on one stream: each has its own scratch, so
    their launches may interleave."""
    import threading
    cases = [make(300, 264, 136, "bf16", 20 + i) for i in range(4)]
    on_gpu = [{k: v.cuda() for k, v in d.items()} for d in cases]

    def call(d):
        return b2.linear_grad(d["dy"], d["x"], d["w"], d["z"], activation=2)
    want = [call(d) for d in on_gpu]
    torch.cuda.synchronize()
    wrong, errors = [], []

    def work(i):
        try:
            for _ in range(50):
                got = call(on_gpu[i])
                same = [torch.equal(g, w) for g, w in zip(got, want[i])]
                if not all(same):
                    wrong.append((i, same))
        except Exception as e:  # noqa: BLE001
            errors.append(e)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors and not wrong

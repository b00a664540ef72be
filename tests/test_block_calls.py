"""GPU: the head and gated entry points as programs call them: streams of their own and of
other devices, several threads, programmatic dependent launch off, memory kept until a side
stream has passed, and waits that give up."""
import threading
import time

import pytest
import torch

import residual_add_normalization_gb300 as b2

pytestmark = pytest.mark.gpu

OK, TIMEOUT = 0, 5
EMPTY, DRAINED = 1, 4
LIMIT_NS = 20_000_000
MIB = 1 << 20


class OtherDevice:
    """A stream of the second GPU."""
    device = torch.device("cuda", 1)
    cuda_stream = 0


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def everything(seed, t=torch.bfloat16, tokens=90):
    """A function that runs each entry once on inputs of its own."""
    g = gen(seed)
    rows = torch.randn(tokens, 12, 64, generator=g, device="cuda").to(t)
    q, k = rows[:, :8], rows[:, 8:10]
    gamma = torch.randn(64, generator=g, device="cuda").to(t)
    p, f = torch.arange(tokens, device="cuda"), b2.rotary_frequencies(64)
    x = torch.randn(tokens, 200, generator=g, device="cuda").to(t)
    w = (torch.randn(2 * 72, 200, generator=g, device="cuda") * 0.1).to(t)
    odd = (torch.randn(2 * 33, 200, generator=g, device="cuda") * 0.1).to(t)

    def run(stream=None):
        kw = {} if stream is None else {"stream": stream}
        out = list(b2.rotary(q, k, p, f, inverse=True, **kw))
        out += b2.head_rms_rotary(q, k, gamma, gamma, p, f, interleaved=True, **kw)
        out += b2.head_rms_rotary_grad(q, k, q, k, gamma, gamma, p, f, **kw)
        for weight in (w, odd):
            h, z = b2.gated_linear(x, weight, want_z=True, **kw)
            out += [h, z, *b2.gated_linear_grad(h, x, weight, z, **kw)]
        return out
    return run


def test_a_stream_of_another_device_is_refused():
    x, w = torch.ones(4, 8, device="cuda"), torch.ones(16, 8, device="cuda")
    q, z = torch.ones(4, 2, 8, device="cuda"), torch.ones(4, 16, device="cuda")
    p, f = torch.arange(4, device="cuda"), b2.rotary_frequencies(8)
    st = OtherDevice()
    for call in (lambda: b2.rotary(q, q, p, f, stream=st),
                 lambda: b2.head_rms_rotary(q, q, w[0], w[0], p, f, stream=st),
                 lambda: b2.head_rms_rotary_grad(q, q, q, q, w[0], w[0], p, f, stream=st),
                 lambda: b2.gated_linear(x, w, stream=st),
                 lambda: b2.gated_linear_grad(x, x, w, z, stream=st)):
        with pytest.raises(ValueError, match="cuda:1"):
            call()


@pytest.mark.parametrize("t", [torch.bfloat16, torch.float32])
def test_threads_on_streams_of_their_own_and_on_one(t):
    """The scratch of the gradients and of unaligned operands is a thread's own: threads on one
    stream do not share it either."""
    runs = [everything(seed, t) for seed in range(4)]
    want = [run() for run in runs]
    torch.cuda.synchronize()
    shared = torch.cuda.Stream()
    for streams in ([torch.cuda.Stream() for _ in runs], [shared] * len(runs)):
        got, errors = [None] * len(runs), []

        def worker(i, streams=streams, got=got, errors=errors):
            try:
                with torch.cuda.stream(streams[i]):
                    for _ in range(10):
                        out = runs[i]()
                streams[i].synchronize()
                got[i] = out
            except Exception as e:  # noqa: BLE001 -- reported below
                errors.append(e)
        threads = [threading.Thread(target=worker, args=(i,)) for i in range(len(runs))]
        for th in threads:
            th.start()
        for th in threads:
            th.join(120)
        assert not errors, errors
        for a, b in zip(got, want):
            assert all(torch.equal(v, w) for v, w in zip(a, b))


def test_dependent_launch_changes_nothing():
    run = everything(9)
    want = run()
    lib = b2.library()
    assert lib.b200norm_testing_set_pdl(0) == OK
    try:
        got = run()
        torch.cuda.synchronize()
    finally:
        assert lib.b200norm_testing_set_pdl(1) == OK
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("t,rows,n_in,n_out", [
    (torch.bfloat16, 300, 264, 136), (torch.float16, 520, 1024, 520),
    (torch.float32, 300, 520, 520), (torch.bfloat16, 4100, 512, 520),
    (torch.bfloat16, 130, 77, 65), (torch.float32, 40, 64, 36)])
def test_gradients_one_after_another(t, rows, n_in, n_out):
    """The launches of a gradient that run side by side: calls on end whose inputs the launch
    before has just written, whose results the next reads and whose workspace is one, against
    the same with every launch waiting for the one before it; eager and replayed."""
    g, lib = gen(12), b2.library()
    xs = [torch.randn(rows, n_in, generator=g, device="cuda").to(t) for _ in range(6)]
    w = (torch.randn(2 * n_out, n_in, generator=g, device="cuda") * 0.05).to(t)
    dh = torch.randn(rows, n_out, generator=g, device="cuda").to(t)
    x, ws = torch.empty_like(xs[0]), torch.empty(64 * MIB, dtype=torch.uint8, device="cuda")

    def run():
        out = []
        for v in xs:
            x.copy_(v)
            h, z = b2.gated_linear(x, w, want_z=True, workspace=ws)
            dx, dw, db = b2.gated_linear_grad(dh, x, w, z, workspace=ws)
            # the results, read by the next launches
            out += [dx, dw, db, *b2.gated_linear_grad(h, dx, w, z, workspace=ws)]
            _, dwl, dbl = b2.linear_grad(z, dx, dw, workspace=ws)
            out += [dwl, dbl]
        return out

    assert lib.b200norm_testing_set_pdl(0) == OK
    try:
        want = run()
        torch.cuda.synchronize()
    finally:
        assert lib.b200norm_testing_set_pdl(1) == OK
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(run(), want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = run()
    for _ in range(3):
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    b2.linear_status()


def test_a_side_stream_s_calls():
    run = everything(10)
    want = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = run(side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("entry", ["rotary", "head_rms_rotary_grad", "gated_linear",
                                   "gated_linear_grad"])
def test_outputs_and_workspace_stay_until_the_stream_has_passed(entry):
    """The caller's outputs and workspace, let go of right after the call, are not handed out
    again while the call is still ahead on a side stream."""
    n = 2048
    q = torch.ones(n // 8, 8, n, device="cuda")[..., :1024].contiguous()
    x, w = torch.ones(n, n // 2, device="cuda"), torch.ones(2 * n, n // 2, device="cuda")
    z = torch.ones(n, 2 * n, device="cuda")
    dh = torch.ones(n, n, device="cuda")
    gamma = torch.ones(1024, device="cuda")
    p, f = torch.arange(n // 8, device="cuda"), b2.rotary_frequencies(64)
    side = torch.cuda.Stream()
    shapes = {"rotary": [q.shape, q.shape], "head_rms_rotary_grad": [q.shape, q.shape],
              "gated_linear": [dh.shape, z.shape], "gated_linear_grad": [x.shape, w.shape]}[entry]
    outs = [torch.empty(s, device="cuda") for s in shapes]
    ws = torch.empty(128 * MIB, dtype=torch.uint8, device="cuda")
    calls = {
        "rotary": lambda: b2.rotary(q, q, p, f, q_out=outs[0], k_out=outs[1], stream=side),
        "head_rms_rotary_grad": lambda: b2.head_rms_rotary_grad(
            q, q, q, q, gamma, gamma, p, f, dq_out=outs[0], dk_out=outs[1], workspace=ws,
            stream=side),
        "gated_linear": lambda: b2.gated_linear(x, w, h=outs[0], z=outs[1], stream=side),
        "gated_linear_grad": lambda: b2.gated_linear_grad(dh, x, w, z, dx=outs[0], dw=outs[1],
                                                          workspace=ws, stream=side),
    }
    call = calls[entry]
    call()  # the kernels are loaded
    torch.cuda.synchronize()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)  # about a tenth of a second ahead of the call
    call()
    used = {t.data_ptr() for t in outs}
    if entry.endswith("grad"):
        used.add(ws.data_ptr())
    outs.clear()
    del ws, call, calls
    again = [torch.empty(s, device="cuda") for s in shapes]
    again.append(torch.empty(128 * MIB, dtype=torch.uint8, device="cuda"))
    assert not side.query()  # the call is still ahead
    assert not used & {t.data_ptr() for t in again}
    torch.cuda.synchronize()


@pytest.fixture
def normal_launches():
    yield
    lib = b2.library()
    lib.b200norm_testing_linear_withhold(0, 0)
    lib.b200norm_testing_force_linear(0, 0, 0, 0)
    b2.linear_status()


MANY = (2600, 136, 2184)


@pytest.mark.parametrize("keep", [False, True])
@pytest.mark.parametrize("site,tiling,shape", [
    (EMPTY, (2, 256, 1, 0), MANY), (EMPTY, (1, 128, 1, 0), MANY),
    (EMPTY, (1, 128, 4, 0), (100, 4096, 200)), (EMPTY, (1, 16, 2, 1), (9, 2048, 300)),
    (EMPTY, (1, 16, 1, 1), (9, 2048, 300)),
    (DRAINED, (2, 256, 1, 0), MANY), (DRAINED, (1, 128, 1, 0), MANY)])
def test_each_wait_of_a_gated_product_gives_up(normal_launches, site, tiling, shape, keep):
    rows, n_in, n_out = shape
    lib = b2.library()
    g = gen(1)
    x, w = (torch.randn(*s, generator=g, device="cuda").bfloat16()
            for s in ((rows, n_in), (2 * n_out, n_in)))
    assert lib.b200norm_testing_force_linear(*tiling) == OK
    want = b2.gated_linear(x, w, want_z=keep)
    b2.linear_status()
    assert lib.b200norm_testing_linear_withhold(site, LIMIT_NS) == OK
    t0 = time.monotonic()
    b2.gated_linear(x, w, want_z=keep)
    with pytest.raises(b2.B200NormError, match=f"wait {site} gave up") as e:
        b2.linear_status()
    assert e.value.status == TIMEOUT
    assert time.monotonic() - t0 < 5.0
    b2.linear_status()  # read and cleared
    assert lib.b200norm_testing_linear_withhold(0, 0) == OK
    got = b2.gated_linear(x, w, want_z=keep)
    b2.linear_status()
    assert torch.equal(got[0], want[0]) and (not keep or torch.equal(got[1], want[1]))

"""A stream of the caller's own: it has to be of the tensors' device, and what the
caller passes stays allocated until the stream has passed the call."""
import pytest
import torch

import residual_add_normalization_gb300 as b2


class OtherDevice:
    """A stream of the second GPU."""
    device = torch.device("cuda", 1)
    cuda_stream = 0


class Tensor(torch.Tensor):
    """Counts what is recorded."""
    recorded = 0

    @property
    def is_cuda(self):
        return True

    def record_stream(self, stream):
        Tensor.recorded += 1


def test_a_stream_of_another_device_is_refused_first():
    Tensor.recorded = 0
    with pytest.raises(ValueError, match="cuda:1"):
        b2._on(0, OtherDevice(), (torch.zeros(2).as_subclass(Tensor), None))
    assert Tensor.recorded == 0


@pytest.mark.gpu
def test_each_entry_refuses_a_stream_of_another_device():
    x, w = torch.ones(4, 8, device="cuda"), torch.ones(8, 8, device="cuda")
    e = torch.ones(4, 1, device="cuda")
    st = OtherDevice()
    for call in (lambda: b2.skip_layer(x, x, w[0], stream=st),
                 lambda: b2.skip_layer_stats(x, x, w[0], stream=st),
                 lambda: b2.skip_layer_grad(x, x, e, e, w[0], stream=st),
                 lambda: b2.linear(x, w, stream=st),
                 lambda: b2.linear_grad(x, x, w, stream=st)):
        with pytest.raises(ValueError, match="cuda:1"):
            call()


def test_the_older_entries_helper_refuses_it_too():
    with pytest.raises(ValueError, match="cuda:1"):
        b2._stream(torch.device("cuda", 0), OtherDevice())
    assert b2._stream(torch.device("cuda", 1), OtherDevice()).value is None
    assert b2._stream("cuda", OtherDevice()).value is None


@pytest.mark.gpu
def test_each_older_entry_refuses_a_stream_of_another_device():
    x, w = torch.ones(4, 8, device="cuda"), torch.ones(8, device="cuda")
    x4 = torch.ones(1, 2, 2, 8, device="cuda")
    st = OtherDevice()
    for call in (lambda: b2.skip_rms(x, x, w, stream=st),
                 lambda: b2.skip_rms_stats(x, x, w, stream=st),
                 lambda: b2.gated_rms(x, x, w, stream=st),
                 lambda: b2.skip_group(x4, x4, w, w, groups=2, activation=0, stream=st)):
        with pytest.raises(ValueError, match="cuda:1"):
            call()


MIB = 1 << 20


@pytest.mark.gpu
@pytest.mark.parametrize("entry", ["skip_layer", "skip_layer_grad", "linear", "linear_grad"])
def test_dropped_outputs_and_workspace_are_not_reused_at_once(entry):
    """Outputs and workspace that the caller drops right after the call: while the
    call's stream still has it ahead, an allocation of the same size on another
    stream does not get their memory."""
    n = 1024  # 4 MiB tensors: blocks of their own size in the caching allocator
    x = torch.ones(n, n, device="cuda")
    e = torch.ones(n, 1, device="cuda")
    vec = x[0].contiguous()
    side = torch.cuda.Stream()

    def big():
        return torch.empty(n, n, device="cuda")
    ws = torch.empty(64 * MIB, dtype=torch.uint8, device="cuda")
    outs = [big(), big()]
    calls = {
        "skip_layer": lambda: b2.skip_layer(x, x, vec, output=outs[0], sum_out=outs[1],
                                            stream=side),
        "skip_layer_grad": lambda: b2.skip_layer_grad(x, x, e, e, vec, dx=outs[0], workspace=ws,
                                                      stream=side),
        "linear": lambda: b2.linear(x, x, y=outs[0], z=outs[1], stream=side),
        "linear_grad": lambda: b2.linear_grad(x, x, x, dx=outs[0], dw=outs[1], workspace=ws,
                                              stream=side),
    }
    call = calls[entry]
    call()  # the kernels are loaded
    torch.cuda.synchronize()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)  # about a tenth of a second ahead of the call
    call()
    used = {t.data_ptr() for t in outs}
    if entry.startswith("skip_layer_grad"):
        used.discard(outs[1].data_ptr())
    if entry.endswith("grad"):
        used.add(ws.data_ptr())
    outs.clear()
    del ws, call, calls
    again = [big() for _ in range(2)]
    again.append(torch.empty(64 * MIB, dtype=torch.uint8, device="cuda"))
    assert not side.query()  # the call is still ahead
    assert not used & {t.data_ptr() for t in again}
    torch.cuda.synchronize()


@pytest.mark.gpu
@pytest.mark.parametrize("given", [False, True])
def test_no_scratch_is_kept_for_a_stream_made_elsewhere(given):
    """Its handle may come back for another stream; torch's own streams keep theirs."""
    x, w = torch.randn(300, 1024, device="cuda"), torch.ones(1024, device="cuda")
    y, s, mean, inv = b2.skip_layer_stats(x, None, w)
    want = b2.skip_layer_grad(y, s, mean, inv, w)
    made = torch.cuda.Stream()
    key = (x.get_device(), made.cuda_stream)
    for stream in (torch.cuda.ExternalStream(made.cuda_stream), made):
        b2._scratch_of_thread.blocks.pop(key, None)
        stream.wait_stream(torch.cuda.current_stream())
        if given:
            got = b2.skip_layer_grad(y, s, mean, inv, w, stream=stream)
        else:
            with torch.cuda.stream(stream):
                got = b2.skip_layer_grad(y, s, mean, inv, w)
        stream.synchronize()
        assert all(torch.equal(g, v) for g, v in zip(got[:3], want[:3]))
        assert (key in b2._scratch_of_thread.blocks) == (stream is made)

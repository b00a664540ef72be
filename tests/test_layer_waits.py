"""The streamed gradient's wait for the other CTAs' sums of a long row: it is made to
give up on the host's word, the call returns, the status says so once, and the next
call is right."""
import time

import pytest
import torch

import residual_add_normalization_gb300 as b2
from residual_add_normalization_gb300 import buildlib

TIMEOUT, INVALID, OK = 5, 1, 0
LIMIT_NS = 20_000_000


def test_withhold_hook_refusals():
    buildlib.build()
    f = b2.library().b200norm_testing_layer_withhold
    assert f(2, 1000) == INVALID
    assert f(-1, 1000) == INVALID
    assert f(1, 0) == INVALID
    assert f(1, 100_000_001) == INVALID
    assert f(0, 0) == OK


@pytest.fixture
def normal_launches():
    yield
    b2.library().b200norm_testing_layer_withhold(0, 0)
    b2.rows_status()


# two and eight CTAs per row, one row or several per cluster, rows that are not whole
# vectors
@pytest.mark.gpu
@pytest.mark.parametrize("rows,hidden,t", [(300, 16384, torch.bfloat16), (3, 65536, torch.float16),
                                           (100, 32768, torch.float32),
                                           (400, 20001, torch.float16)])
def test_the_wait_for_sums_gives_up(normal_launches, rows, hidden, t):
    lib = b2.library()
    g = torch.Generator(device="cuda").manual_seed(2)
    x, dy = (torch.randn(rows, hidden, generator=g, device="cuda").to(t) for _ in range(2))
    gamma = torch.ones(hidden, device="cuda")
    _, s, mean, inv = b2.skip_layer_stats(x, None, gamma)
    want = b2.skip_layer_grad(dy, s, mean, inv, gamma, want_bias=True)
    b2.rows_status()
    assert lib.b200norm_testing_layer_withhold(1, LIMIT_NS) == OK
    t0 = time.monotonic()
    b2.skip_layer_grad(dy, s, mean, inv, gamma, want_bias=True)
    with pytest.raises(b2.B200NormError) as e:
        b2.rows_status()
    assert e.value.status == TIMEOUT
    assert time.monotonic() - t0 < 2.0
    b2.rows_status()  # read and cleared
    # a row of a CTA's own sends nothing
    small = b2.skip_layer_grad(dy[:, :768].contiguous(), x[:, :768].contiguous(), mean, inv,
                               gamma[:768])
    b2.rows_status()
    assert lib.b200norm_testing_layer_withhold(0, 0) == OK
    got = b2.skip_layer_grad(dy, s, mean, inv, gamma, want_bias=True)
    again = b2.skip_layer_grad(dy[:, :768].contiguous(), x[:, :768].contiguous(), mean, inv,
                               gamma[:768])
    b2.rows_status()
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    assert all(torch.equal(p, q) for p, q in zip(small[:3], again[:3]))

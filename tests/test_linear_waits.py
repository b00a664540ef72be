"""The bounded waits of the linear operator's tensor-core products: each kind is
made to give up on the host's word, the call returns, the status names the kind,
and the next call is right."""
import time

import pytest
import torch

import residual_add_normalization_gb300 as b2
from residual_add_normalization_gb300 import buildlib

TIMEOUT, INVALID, OK = 5, 1, 0
EMPTY, DRAINED, RESIDUAL = 1, 4, 5
LIMIT_NS = 20_000_000


def test_withhold_hook_refusals():
    buildlib.build()
    f = b2.library().b200norm_testing_linear_withhold
    for site in (-1, 2, 3, 6, 100):
        assert f(site, 1000) == INVALID, site
    assert f(EMPTY, 0) == INVALID
    assert f(EMPTY, 100_000_001) == INVALID
    assert f(0, 0) == OK


@pytest.fixture
def normal_launches():
    yield
    lib = b2.library()
    lib.b200norm_testing_linear_withhold(0, 0)
    lib.b200norm_testing_force_linear(0, 0, 0, 0)
    b2.linear_status()


# several tiles per CTA, which reuse a stage and a buffer of sums; K in parts; the
# weight's rows in the lanes
MANY = (2600, 136, 4360)
CASES = [(EMPTY, (2, 256, 1, 0), MANY), (EMPTY, (1, 128, 1, 0), MANY), (EMPTY, (1, 64, 1, 0), MANY),
         (EMPTY, (1, 128, 4, 0), (100, 4096, 200)), (EMPTY, (1, 16, 2, 1), (9, 2048, 300)),
         (DRAINED, (2, 256, 1, 0), MANY), (DRAINED, (1, 128, 1, 0), MANY),
         (DRAINED, (1, 64, 1, 0), MANY),
         (RESIDUAL, (2, 256, 1, 0), MANY), (RESIDUAL, (1, 128, 1, 0), MANY),
         (RESIDUAL, (1, 64, 1, 0), (70, 64, 72))]


@pytest.mark.gpu
@pytest.mark.parametrize("keep", [False, True])
@pytest.mark.parametrize("site,tiling,shape", CASES)
def test_each_wait_gives_up(normal_launches, site, tiling, shape, keep):
    rows, n_in, n_out = shape
    lib = b2.library()
    g = torch.Generator(device="cuda").manual_seed(1)
    x, w, r = (torch.randn(*s, generator=g, device="cuda").bfloat16()
               for s in ((rows, n_in), (n_out, n_in), (rows, n_out)))
    assert lib.b200norm_testing_force_linear(*tiling) == OK

    def call():
        return b2.linear(x, w, None, r, activation=2, want_z=keep)
    want = call()
    b2.linear_status()
    assert lib.b200norm_testing_linear_withhold(site, LIMIT_NS) == OK
    t0 = time.monotonic()
    call()
    with pytest.raises(b2.B200NormError, match=f"wait {site} gave up") as e:
        b2.linear_status()
    assert e.value.status == TIMEOUT
    assert time.monotonic() - t0 < 5.0
    b2.linear_status()  # read and cleared
    assert lib.b200norm_testing_linear_withhold(0, 0) == OK
    got = call()
    b2.linear_status()
    assert torch.equal(got[0], want[0]) and (not keep or torch.equal(got[1], want[1]))

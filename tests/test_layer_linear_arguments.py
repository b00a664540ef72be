"""GPU: epsilon and activation of the layer and linear entries in the forms that the
other operators take: anything that float() and int() take."""
import numpy as np
import pytest
import torch

import residual_add_normalization_gb300 as b2

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("eps", [np.float32(0.5), np.float64(0.5), torch.tensor(0.5),
                                 np.array(0.5)])
def test_epsilon(eps):
    x = torch.randn(3, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    want = b2.skip_layer_stats(x, x, w, epsilon=0.5)
    got = b2.skip_layer_stats(x, x, w, epsilon=eps)
    assert all(torch.equal(g, v) for g, v in zip(got, want))
    assert torch.equal(b2.skip_layer(x, x, w, epsilon=eps)[0], want[0])
    b2.skip_rms(x, x, w, epsilon=eps)  # as the older entries do


@pytest.mark.parametrize("act", [np.int64(2), np.int32(2), torch.tensor(2), 2.0])
def test_activation(act):
    x, w = torch.randn(3, 64, device="cuda"), torch.randn(8, 64, device="cuda")
    y, z = b2.linear(x, w, activation=2, want_z=True)
    assert torch.equal(b2.linear(x, w, activation=act)[0], y)
    want = b2.linear_grad(y, x, w, z, activation=2)
    got = b2.linear_grad(y, x, w, z, activation=act)
    assert all(torch.equal(g, v) for g, v in zip(got, want))
    x4 = torch.ones(1, 2, 2, 8, device="cuda")
    b2.skip_group(x4, x4, x4[0, 0, 0], x4[0, 0, 0], groups=2, activation=type(act)(1)
                  if not isinstance(act, torch.Tensor) else torch.tensor(1))


def test_none_of_them():
    x, w = torch.randn(3, 64, device="cuda"), torch.randn(8, 64, device="cuda")
    with pytest.raises(ValueError):
        b2.linear(x, w, activation="gelu")
    with pytest.raises(b2.B200NormError):
        b2.linear(x, w, activation=np.int64(5))

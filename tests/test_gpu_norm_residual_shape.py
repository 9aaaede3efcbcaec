"""GPU test of the layer norm's autograd wrapper with a residual whose leading dimensions are others
than x's: each gradient has its input's shape."""
import pytest
import torch

from test_gpu_norm import EPS, b, draw  # noqa: F401

pytestmark = pytest.mark.gpu
F32 = torch.float32


@pytest.mark.parametrize("use", ["y", "s", "both"])
def test_a_residual_of_another_shape_gets_its_own_back(b, use):  # noqa: F811
    """x [2, 9, D] with a residual given as [18, D]: each gradient has its input's shape."""
    t = draw(18, 136, F32, F32, seed=3)
    x, r = t["x"].reshape(2, 9, 136).clone().requires_grad_(), t["r"].clone().requires_grad_()
    y, s = b.layer_norm(x, t["gamma"], t["beta"], EPS, residual=r)
    assert y.shape == s.shape == x.shape
    ((y * t["dy"].reshape(2, 9, 136)).sum() * (use != "s") + s.sin().sum() * (use != "y")).backward()
    assert x.grad.shape == x.shape and r.grad.shape == r.shape
    assert torch.equal(x.grad.reshape(18, 136), r.grad)
    assert x.grad.data_ptr() != r.grad.data_ptr(), "each gradient can be scaled in its place"


def test_the_sum_alone(b):  # noqa: F811
    """No gradient reaches y: s passes its own on, in both shapes."""
    t = draw(18, 136, F32, F32, seed=4)
    x, r = t["x"].reshape(2, 9, 136).clone().requires_grad_(), t["r"].clone().requires_grad_()
    _, s = b.layer_norm(x, t["gamma"], t["beta"], EPS, residual=r)
    s.sin().sum().backward()
    assert torch.equal(x.grad, s.detach().cos()) and torch.equal(r.grad, x.grad.reshape(18, 136))


@pytest.mark.parametrize("shape", [(18, 136), (2, 9, 136)])
@pytest.mark.parametrize("use", ["y", "s"])
def test_the_gradients_are_tensors_of_their_own(b, shape, use):  # noqa: F811
    """x's gradient scaled in place leaves the residual's as it is."""
    t = draw(18, 136, F32, F32, seed=5)
    x, r = t["x"].reshape(shape).clone().requires_grad_(), t["r"].reshape(shape).clone().requires_grad_()
    y, s = b.layer_norm(x, t["gamma"], t["beta"], EPS, residual=r)
    (y if use == "y" else s).sin().sum().backward()
    kept = r.grad.clone()
    x.grad.zero_()
    assert torch.equal(r.grad, kept) and bool(kept.any())

"""GPU tests of the autograd wrappers: second derivatives, which the backward kernels do not have, are
refused however they are asked for; a graph of the first (create_graph) changes nothing."""
import pytest
import torch

from test_gpu_norm import EPS, b, draw  # noqa: F401

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def norm_inputs():
    t = draw(6, 64, F32, F32, seed=1)
    return [t[k].clone().requires_grad_() for k in ("x", "gamma", "beta", "r")]


def block_inputs():
    g = torch.Generator().manual_seed(2)
    return [torch.randn(*s, generator=g).to(BF).cuda().requires_grad_() for s in ((16, 64), (128, 64), (64, 64))]


def calls(b):  # noqa: F811
    return {
        "norm": (norm_inputs, lambda x, w, c, r: b.layer_norm(x, w, c, EPS)[0]),
        "norm without parameters": (norm_inputs, lambda x, w, c, r: b.layer_norm(x, None, None, EPS)[0]),
        "norm of a view": (norm_inputs, lambda x, w, c, r: b.layer_norm(x.reshape(2, 3, 64), w, c, EPS)[0]),
        "norm with a residual": (norm_inputs, lambda x, w, c, r: b.layer_norm(x, w, c, EPS, residual=r)[0]),
        "its sum": (norm_inputs, lambda x, w, c, r: sum(v.sin() for v in b.layer_norm(x, w, c, EPS, residual=r))),
        "block": (block_inputs, lambda x, W1, W2: b.swiglu_mlp(x, W1, W2).float()),
        "residual block": (block_inputs, lambda x, W1, W2: b.swiglu_mlp(x, W1, W2, True).float()),
    }


NAMES = ["norm", "norm without parameters", "norm of a view", "norm with a residual", "its sum", "block", "residual block"]


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("loss", ["linear", "quadratic"])
def test_a_second_derivative_is_refused(b, name, loss):  # noqa: F811
    """A gradient penalty would lose its terms through the kernel without a word."""
    make, f = calls(b)[name]
    inputs = make()
    x, y = inputs[0], f(*inputs)
    gx, = torch.autograd.grad(y.sum() if loss == "linear" else y.square().sum(), x, create_graph=True)
    penalty = gx.float().square().sum() + x.float().sum()
    with pytest.raises(RuntimeError, match="not differentiable"):
        torch.autograd.grad(penalty, x, retain_graph=True)
    with pytest.raises(RuntimeError, match="not differentiable"):
        penalty.backward()


@pytest.mark.parametrize("name", NAMES)
def test_the_first_derivative_is_the_same_with_a_graph(b, name):  # noqa: F811
    make, f = calls(b)[name]
    first, second = make(), make()
    g0 = torch.autograd.grad(f(*first).square().sum(), first, allow_unused=True)
    g1 = torch.autograd.grad(f(*second).square().sum(), second, allow_unused=True, create_graph=True)
    for p, q in zip(g0, g1):
        assert (p is None) == (q is None) and (p is None or torch.equal(p, q))

"""GPU tests of the gradient clipping where squares overflow fp32 (tolerances: test_gpu_clip.py)."""
import pytest
import torch

from test_gpu_clip import BF, F32, U, b, grads_of, norm64  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("scale", [1e17, 1e18, 1e19, 1e25, 1e32, 3e34])
def test_large_gradients(b, scale):  # noqa: F811
    """Elements up to 5 deviations; the norm itself stays within fp32."""
    grads = grads_of([(40000, BF), (999, F32), (70001, F32), (3, BF)], 13, std=scale)
    want = norm64(grads)
    assert abs(b.swiglu_mlp_grad_norm(grads).item() - want) <= 12 * U * want


def test_one_large_element_among_small_ones(b):  # noqa: F811
    for big in (1e19, 2e19, 3e38):
        t = grads_of([(50000, F32)], 14, std=1e-20)[0]
        t[777] = big
        assert abs(b.swiglu_mlp_grad_norm([t]).item() - norm64([t])) <= 12 * U * norm64([t])

"""GPU tests of the gradient clipping where squares fall below fp32's normal range.

Tolerances: those of test_gpu_clip.py, 12 u for the norm, hold down to the smallest elements a type
has, since sums too small for fp32 are taken again of scaled elements."""
import pytest
import torch

from test_gpu_clip import BF, F32, HF, TINY, U, UT, b, grads_of, norm64  # noqa: F401

pytestmark = pytest.mark.gpu
LIST = [(40000, BF), (999, F32), (70001, F32), (3, BF), (17, F32), (16385, BF)]


@pytest.mark.parametrize("scale", [1e-17, 1e-18, 1e-19, 1e-20, 1e-22, 3e-23, 1e-25, 1e-32])
def test_small_gradients(b, scale):  # noqa: F811
    grads = grads_of(LIST, 11, std=scale)
    want = norm64(grads)
    norm = b.swiglu_mlp_grad_norm(grads)
    assert abs(norm.item() - want) <= 12 * U * want
    for max_norm in (scale, 1.0):
        factor = min(1.0, max_norm / want)
        norm, got = b.swiglu_mlp_clip_grads(grads, max_norm, 0.0, out=[torch.empty_like(t) for t in grads])
        assert abs(norm.item() - want) <= 12 * U * want
        for p, q in zip(got, grads):
            ref = q.double() * factor
            # the C entry takes max_norm in fp32, and an output is rounded once
            assert bool(((p.double() - ref).abs() <= ref.abs() * (UT[p.dtype] + 25 * U) + TINY[p.dtype]).all())


def test_small_beside_large_and_zero(b):  # noqa: F811
    """A few small elements in a block of zeros count; beside large ones they change nothing."""
    t = torch.zeros(50000, device="cuda")
    t[[3, 20000, 49999]] = torch.tensor([3e-25, 4e-25, 12e-25], device="cuda")
    assert abs(b.swiglu_mlp_grad_norm([t]).item() - 13e-25) <= 13e-25 * 12 * U
    big = torch.full((50000,), 2.0, device="cuda")
    both = norm64([t, big])
    assert abs(b.swiglu_mlp_grad_norm([t, big, torch.zeros(9999, dtype=HF, device="cuda")]).item() - both) <= 12 * U * both
    smallest = torch.full((30000,), 2.0 ** -149, device="cuda")
    assert abs(b.swiglu_mlp_grad_norm([smallest]).item() - norm64([smallest])) <= 2.0 ** -150 + 12 * U * norm64([smallest])
    assert b.swiglu_mlp_grad_norm([torch.zeros(70000, device="cuda"), torch.zeros(5, dtype=BF, device="cuda")]).item() == 0.0

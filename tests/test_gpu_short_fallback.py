"""GPU test of the operators' calls where the compiled module is missing: the same bits by ctypes."""
import pytest
import torch

from test_gpu_short_calls import BF, F32, b, z  # noqa: F401

pytestmark = pytest.mark.gpu


def test_the_same_without_the_module(b, monkeypatch):  # noqa: F811
    x, r, w = z(37, 200), z(37, 200) * 2, z(200, dtype=F32)
    W = z(37, 64), z(6, 64), z(6, 128, 64), z(6, 64, 64)

    def calls():
        y, s, mean, rstd = b.swiglu_mlp_layer_norm_fwd(x, w, w, 1e-5, residual=r)
        grads = b.swiglu_mlp_layer_norm_bwd(r, s, w, mean, rstd, dskip=x)
        norm, out = b.swiglu_mlp_clip_grads([g.clone() for g in grads], 0.5)
        return (y, s, mean, rstd, *grads, norm, *out, b.swiglu_mlp_grad_norm([x, w]), *b.swiglu_moe_routed_fwd(*W, 2))

    want = calls()
    monkeypatch.setattr(b, "_short_calls", b._NoShortCalls())
    assert all(torch.equal(p, q) for p, q in zip(calls(), want))

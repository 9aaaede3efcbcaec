"""GPU tests of the layer norm on rows of millions of columns, against fp64.

The tolerances are those of test_gpu_norm.py, which bound a row sum by 53 u (u = 2^-24) of the sum of
magnitudes whatever the width: a thread's long sum is taken in runs of at most 32 elements, whose
sums are added with their rounding errors kept, so it is off by 32 u, and 16 warps' sums follow in
9 steps.  Values away from 0 make every rounding of a plain running sum lean the same way."""
import pytest
import torch

from test_gpu_norm import EPS, b, check_bwd, check_fwd  # noqa: F401

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def rows(M, D, dtype, seed, mean=1.1, dev=0.1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.empty(M, D, device="cuda").normal_(mean, dev, generator=g).to(dtype)


# 16-byte packs of fp32 and bf16; single elements
@pytest.mark.parametrize("D,dtype", [(2 ** 24 + 4, F32), (2 ** 24 + 8, BF), (2 ** 22 + 1, F32)])
@pytest.mark.parametrize("residual", [False, True])
def test_long_rows(b, D, dtype, residual):  # noqa: F811
    x, r = rows(2, D, dtype, 1), rows(2, D, dtype, 2) if residual else None
    _, s, mean, rstd = check_fwd(b, None, x, r, None, None)
    check_bwd(b, rows(2, D, dtype, 3), s, None, mean, rstd, r, param_grads=False)


def test_a_long_constant_row(b):  # noqa: F811
    """mean is the value, so y is beta and rstd 1 / sqrt(eps)."""
    x = torch.full((1, 2 ** 24), 1.1, device="cuda")
    y, _, mean, rstd = b.swiglu_mlp_layer_norm_fwd(x, None, None, EPS)
    assert abs(mean.item() - x[0, 0].item()) <= 54 * 2 ** -24 * 1.1
    assert abs(rstd.item() * EPS ** 0.5 - 1) <= 1e-5
    assert y.abs().max().item() <= 54 * 2 ** -24 * 1.1 * EPS ** -0.5 * 1.01


@pytest.mark.parametrize("D", [40000, 40001])
def test_infinities_and_nan_in_rows_past_the_registers(b, D):  # noqa: F811
    x = rows(4, D, BF, 5)
    x[1, 17], x[2, D - 1] = float("inf"), float("nan")
    y, _, mean, rstd = b.swiglu_mlp_layer_norm_fwd(x, None, None, EPS)
    clean = b.swiglu_mlp_layer_norm_fwd(rows(4, D, BF, 5), None, None, EPS)
    assert mean[1].item() == float("inf") and bool(mean[2].isnan()) and bool(rstd[1:3].isnan().all())
    assert bool(y[1:3].isnan().all()) and torch.equal(y[::3], clean[0][::3])

"""GPU tests of the layer norm's backward on rows whose mean is far from 0, against fp64.

Tolerances (u = 2^-24; sums and roundings as in test_gpu_norm.py).  The saved statistics are taken as
given, so xh = (s - mean) * rstd is two roundings: 2 u of |xh|, whatever the mean.  dx then stays
within 200 u of the magnitudes of its three terms, and a column sum of M rows and at most 100 partial
sums within (M + 100) u of the sum of |dy xh|."""
import pytest
import torch

from test_gpu_norm import EPS, U, b, draw, within  # noqa: F401

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32

# (M, D, row offset): whole packs, one row a group and several; shifted packs; element by element
# (few rows; rows that lie differently; a narrow row); rows in two passes, packs and elements
FORMS = [(40, 2048, 0), (700, 3584, 0), (5, 6144, 0), (700, 1021, 0), (1537, 5003, 1), (40, 1021, 0), (1000, 31, 0),
         (40, 8192, 0), (12, 8195, 0)]


@pytest.mark.parametrize("M,D,off", FORMS)
@pytest.mark.parametrize("dtype,ratio", [(F32, 1000.0), (F32, 30.0), (BF, 64.0)])
def test_mean_far_from_zero(b, M, D, off, dtype, ratio):  # noqa: F811
    t = draw(M, D, F32, F32, seed=M + D, shift=0.0)

    def place(v):
        flat = torch.empty(M * D + 16, dtype=dtype, device="cuda")[off:off + M * D].view(M, D)
        return flat.copy_(v)

    s, dy, skip = place(1.0 + t["x"] / ratio), place(t["dy"]), place(t["ds"] / 8)
    _, _, mean, rstd = b.swiglu_mlp_layer_norm_fwd(s, t["gamma"], t["beta"], EPS * ratio ** -2)
    for k in (None, skip):
        dx, dgamma, dbeta = b.swiglu_mlp_layer_norm_bwd(dy, s, t["gamma"], mean, rstd, dskip=k)
        d, rs = dy.double(), rstd.double()[:, None]
        xh, g = (s.double() - mean.double()[:, None]) * rs, d * t["gamma"].double()
        ref = rs * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
        scale = 200 * U * rs * (g.abs() + g.abs().mean(1, keepdim=True) + xh.abs() * (g * xh).abs().mean(1, keepdim=True))
        if k is not None:
            ref = ref + k.double()
            scale = scale + U * ref.abs()
        within(dx, ref, scale, "dx")
        within(dgamma, (d * xh).sum(0), (M + 100) * U * (d * xh).abs().sum(0), "dgamma")
        within(dbeta, d.sum(0), (M + 100) * U * d.abs().sum(0), "dbeta")

"""GPU tests of the layer norm's last pair of types, fp16 rows with fp32 parameters, in every form of
its rows (tolerances: test_gpu_norm.py)."""
import pytest
import torch

from test_gpu_norm import EPS, b, check_bwd, check_fwd, draw  # noqa: F401
from test_gpu_norm_rows import run

pytestmark = pytest.mark.gpu
HF, F32 = torch.float16, torch.float32


@pytest.mark.parametrize("M,D", [(1, 1), (3, 7), (33, 256), (300, 1032), (9, 3584), (3, 8192), (2, 12288), (3, 16384),
                                 (2, 40000), (700, 515), (5000, 24)])
def test_whole_rows(b, M, D):  # noqa: F811
    t = draw(M, D, HF, F32, seed=D)
    for r, skip in ((None, None), (t["r"], t["ds"])):
        _, s, mean, rstd = check_fwd(b, t, t["x"], r, t["gamma"], t["beta"])
        check_bwd(b, t["dy"], s, t["gamma"], mean, rstd, skip)


@pytest.mark.parametrize("M,D,off", [(700, 129, 1), (401, 1021, 7), (310, 4091, 0), (3, 12290, 3), (2, 33001, 1), (152, 5003, 2)])
@pytest.mark.parametrize("residual", [False, True])
def test_rows_off_16_bytes(b, M, D, off, residual):  # noqa: F811
    run(b, M, D, HF, F32, off, residual)


@pytest.mark.parametrize("D", [61, 2050, 9001])
def test_rows_that_lie_differently(b, D):  # noqa: F811
    run(b, 40, D, HF, F32, 1, True, offs=[1, 2, 3, 2])


@pytest.mark.parametrize("D", [64, 8192])
def test_parameters_off_16_bytes(b, D):  # noqa: F811
    run(b, 20, D, HF, F32, 0, True, poff=1)

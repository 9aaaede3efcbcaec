"""GPU tests of the layer norm on rows that lie off 16-byte boundaries, alike in every tensor or
not, and on the widest rows of each form, against fp64 (tolerances: test_gpu_norm.py)."""
import pytest
import torch

from test_gpu_norm import U, b, check_bwd, check_fwd, draw  # noqa: F401

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def shifted(v, off):
    """A contiguous copy of v whose first element lies `off` elements past a 16-byte boundary,
    with NaN before and after it."""
    n = v.numel()
    flat = torch.full((n + off + 16,), float("nan"), dtype=v.dtype, device=v.device)
    flat[off:off + n] = v.reshape(-1)
    return flat[off:off + n].view(v.shape), flat


def run(b, M, D, dtype, wdtype, off, residual, offs=None, poff=0):  # noqa: F811
    t = draw(M, D, dtype, wdtype, seed=D + off)
    o = offs or [off] * 4
    x, r, dy, ds = (shifted(t[k], i)[0] for k, i in zip(("x", "r", "dy", "ds"), o))
    gamma, beta = shifted(t["gamma"], poff)[0], shifted(t["beta"], poff)[0]
    (y, whole_y), (s, whole_s), (dx, whole_dx) = (shifted(torch.zeros_like(t["x"]), o[0]) for _ in range(3))
    kw = dict(s=s) if residual else {}
    y, s, mean, rstd = check_fwd(b, t, x, r if residual else None, gamma, beta, y=y, **kw)
    check_bwd(b, dy, s, gamma, mean, rstd, ds if residual else None, dx=dx)
    for name, whole in (("y", whole_y), ("dx", whole_dx)) + ((("s", whole_s),) if residual else ()):
        n = M * D
        assert bool(whole[:o[0]].isnan().all()) and bool(whole[o[0] + n:].isnan().all()), f"{name}: written past its rows"
        assert not bool(whole[o[0]:o[0] + n].isnan().any()), f"{name}: a neighbour's NaN"


# every way a row can start in its pack, many rows a group; widths at the ends of each plan
@pytest.mark.parametrize("M,D", [(1, 65), (2, 64), (1000, 67), (700, 129), (401, 1021), (160, 2043), (310, 4091),
                                 (155, 8189), (3, 12281), (3, 12282), (153, 6141)])
@pytest.mark.parametrize("dtype,wdtype,off", [(BF, BF, 0), (BF, F32, 1), (BF, BF, 7), (F32, F32, 0), (F32, F32, 3)])
@pytest.mark.parametrize("residual", [False, True])
def test_rows_alike(b, M, D, dtype, wdtype, off, residual):  # noqa: F811
    run(b, M, D, dtype, wdtype, off, residual)


@pytest.mark.parametrize("M,D", [(2, 16383), (2, 16389), (2, 29000), (2, 29050), (1, 32768), (2, 32776), (3, 6145), (3, 12290)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_widest_rows(b, M, D, dtype):  # noqa: F811
    run(b, M, D, dtype, F32, 0, True)
    run(b, M, D, dtype, dtype, 3, False)


@pytest.mark.parametrize("D", [61, 515, 2050, 5003, 6131])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_not_alike(b, D, dtype):  # noqa: F811
    run(b, 40, D, dtype, F32, 1, True, offs=[1, 2, 3, 2])


@pytest.mark.parametrize("D", [8, 64, 1024, 3584, 8192, 16384, 32760])
@pytest.mark.parametrize("residual", [False, True])
def test_parameters_off_16_byte_boundaries(b, D, residual):  # noqa: F811
    run(b, 20, D, BF, BF, 0, residual, poff=1)
    run(b, 20, D, BF, F32, 0, residual, poff=1)


def test_rows_in_a_wider_buffer_keep_its_rest(b):  # noqa: F811
    """Row stride off 16 bytes and wider than the rows: what lies between them is neither read
    into the result nor written."""
    M, D, ld = 500, 261, 267
    for dtype in (BF, F32):
        t = draw(M, D, dtype, F32, seed=5)
        wide = {k: torch.full((M, ld), float("nan"), dtype=dtype, device="cuda") for k in ("x", "r", "dy", "ds", "y", "s", "dx")}
        for k in ("x", "r", "dy", "ds"):
            wide[k][:, :D] = t[k]
        v = {k: w[:, :D] for k, w in wide.items()}
        _, s, mean, rstd = check_fwd(b, t, v["x"], v["r"], t["gamma"], t["beta"], y=v["y"], s=v["s"])
        check_bwd(b, v["dy"], s, t["gamma"], mean, rstd, v["ds"], dx=v["dx"])
        for k in ("y", "s", "dx"):
            assert bool(wide[k][:, D:].isnan().all()), k
            assert not bool(v[k].isnan().any()), k


def test_rows_alike_same_bits_and_neighbours(b):  # noqa: F811
    """A row's result does not depend on its neighbours, which share its first and last 16 bytes."""
    M, D = 400, 515
    t = draw(M, D, BF, BF, seed=9)
    a = b.swiglu_mlp_layer_norm_fwd(t["x"], t["gamma"], t["beta"])
    g = b.swiglu_mlp_layer_norm_bwd(t["dy"], t["x"], t["gamma"], a[2], a[3])
    again = b.swiglu_mlp_layer_norm_bwd(t["dy"], t["x"], t["gamma"], a[2], a[3])
    assert all(torch.equal(p, q) for p, q in zip(g, again))
    x, dy = t["x"].clone(), t["dy"].clone()
    x[1::2] = float("nan")
    dy[1::2] = float("inf")
    c = b.swiglu_mlp_layer_norm_fwd(x, t["gamma"], t["beta"])
    h = b.swiglu_mlp_layer_norm_bwd(dy, x, t["gamma"], c[2], c[3])
    for p, q in ((a[0], c[0]), (a[2], c[2]), (a[3], c[3]), (g[0], h[0])):
        assert torch.equal(p[::2], q[::2])

"""GPU tests of the layer norm with an output in an input's place (the residual stream updated where
it stands, a gradient where its source was): the same bits as with outputs of their own."""
import pytest
import torch

from test_gpu_norm import EPS, b, draw  # noqa: F401

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32

# (M, D, type, offsets of x, r, y, s past a 16-byte boundary): whole packs; shifted packs; element by
# element; rows past the registers in packs, off 16 bytes, and lying differently
FORMS = [(20, 1024, BF, (0, 0)), (300, 1021, BF, (0, 0)), (400, 5003, BF, (0, 0)), (20, 515, F32, (0, 0)),
         (30, 700, BF, (1, 2)), (3, 40000, BF, (0, 0)), (3, 40001, BF, (0, 0)), (2, 16392, F32, (0, 0)),
         (3, 9001, BF, (1, 2))]


def at(v, off):
    flat = torch.empty(v.numel() + 16, dtype=v.dtype, device="cuda")
    return flat[off:off + v.numel()].view(v.shape).copy_(v)


@pytest.mark.parametrize("M,D,dtype,offs", FORMS)
@pytest.mark.parametrize("case", ["s=residual", "s=x", "y=x", "y=residual", "s=residual y=x", "y=x alone"])
def test_forward(b, M, D, dtype, offs, case):  # noqa: F811
    t = draw(M, D, dtype, F32, seed=D)
    alone = case.endswith("alone")

    def inputs():
        return at(t["x"], offs[0]), at(t["r"], offs[1])

    x, r = inputs()
    out = dict(y=at(t["x"], offs[0]), s=at(t["r"], offs[1]))
    want = dict(zip(("y", "s", "mean", "rstd"), b.swiglu_mlp_layer_norm_fwd(
        x, t["gamma"], t["beta"], EPS, residual=None if alone else r, **({"y": out["y"]} if alone else out))))
    x, r = inputs()
    places = {"s=residual": dict(s=r), "s=x": dict(s=x), "y=x": dict(y=x), "y=residual": dict(y=r),
              "s=residual y=x": dict(s=r, y=x), "y=x alone": dict(y=x)}[case]
    out = {} if alone else dict(y=at(t["x"], offs[0]), s=at(t["r"], offs[1]))
    got = dict(zip(("y", "s", "mean", "rstd"), b.swiglu_mlp_layer_norm_fwd(
        x, t["gamma"], t["beta"], EPS, residual=None if alone else r, **{**out, **places})))
    same = offs[0] == offs[1] or alone       # another place of a row can mean another order of its sums
    for k in ("y", "mean", "rstd") + (() if alone else ("s",)):
        if same:
            assert torch.equal(got[k], want[k]), k
        else:
            assert (got[k].double() - want[k].double()).abs().max() <= 2 ** -7 * want[k].abs().max(), k


@pytest.mark.parametrize("M,D,dtype,offs", FORMS)
@pytest.mark.parametrize("place", ["dy", "s", "dskip"])
def test_backward(b, M, D, dtype, offs, place):  # noqa: F811
    t = draw(M, D, dtype, F32, seed=D)
    x, dy, ds = (lambda: (at(t["x"], offs[0]), at(t["dy"], offs[1]), at(t["ds"], offs[1])))()
    _, _, mean, rstd = b.swiglu_mlp_layer_norm_fwd(x, t["gamma"], t["beta"], EPS)
    held = {"dy": dy, "s": x, "dskip": ds}
    own = torch.empty_like(held[place])
    own = at(own, offs[0] if place == "s" else offs[1])
    want = b.swiglu_mlp_layer_norm_bwd(dy, x, t["gamma"], mean, rstd, dskip=ds, dx=own)
    got = b.swiglu_mlp_layer_norm_bwd(dy, x, t["gamma"], mean, rstd, dskip=ds, dx=held[place])
    assert got[0] is held[place]
    assert all(torch.equal(p, q) for p, q in zip(got, want))

"""GPU tests of the layer norm (swiglu_mlp_layer_norm_fwd / _bwd) against fp64 torch.

Tolerances.  u = 2^-24 is fp32's unit roundoff, uT the output type's.  A row sum adds at most
16 values a thread, 5 shuffle steps and 32 warps in sequence, so its error is at most 53 u of
the sum of magnitudes; the mean, the variance and the output's own products then stay within
160 u of |gamma| rstd (|s| + mean|s|) + |beta|, and dx within 200 u of the magnitudes of its
three terms.  A column sum adds at most M rows and 100 partial sums.  Each output is rounded
once more to its type.
"""
import pytest
import torch

from helpers import ensure_library

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
UT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: U}
TINY = {torch.bfloat16: 1e-38, torch.float16: 2.0 ** -24, torch.float32: 1e-38}    # below the normal range
EPS = 1e-5


@pytest.fixture(scope="module")
def b():
    ensure_library()
    from bwd_gemm_epilogue_gb300 import binding
    binding.lib()
    return binding


def within(got, ref, scale, what):
    """|got - ref| <= scale + uT |ref| everywhere (ref, scale fp64)."""
    assert got.shape == ref.shape, what
    bound = scale + (UT[got.dtype] * (ref.abs() + scale)) + TINY[got.dtype]
    over = ((got.double() - ref).abs() / bound)
    assert bool((over <= 1).all()), f"{what}: {over.max().item():.3g} times the bound"


def draw(M, D, dtype, wdtype, seed, shift=0.3):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    scale = (0.5 * n(D)).exp()
    t = dict(x=n(M, D) * scale + shift * n(D), r=n(M, D) * scale, dy=n(M, D), ds=n(M, D))
    t = {k: v.to(dtype).cuda() for k, v in t.items()}
    t["gamma"], t["beta"] = ((1 + 0.2 * n(D)).to(wdtype).cuda(), (0.2 * n(D)).to(wdtype).cuda())
    return t


def fwd_ref(s, gamma, beta):
    mean = s.mean(1, keepdim=True)
    rstd = ((s - mean).square().mean(1, keepdim=True) + EPS).rsqrt()
    y = (s - mean) * rstd * gamma + beta
    scale = 160 * U * (gamma.abs() * rstd * (s.abs() + s.abs().mean(1, keepdim=True)) + beta.abs())
    return y, mean, rstd, scale


def check_fwd(b, t, x, r, gamma, beta, **kw):
    y, s, mean, rstd = b.swiglu_mlp_layer_norm_fwd(x, gamma, beta, EPS, residual=r, **kw)
    s64 = x.double() + (0 if r is None else r.double())
    one = torch.ones(x.shape[1], dtype=torch.float64, device="cuda")
    y64, mean64, rstd64, scale = fwd_ref(s64, one if gamma is None else gamma.double(),
                                         0 * one if beta is None else beta.double())
    within(y, y64, scale, "y")
    if r is not None:
        within(s, s64, U * s64.abs(), "s")
    else:
        assert s is x
    mag = s64.abs().mean(1)
    within(mean, mean64[:, 0], 54 * U * mag, "mean")
    within(rstd, rstd64[:, 0], 160 * U * rstd64[:, 0] * (1 + mag * rstd64[:, 0]), "rstd")
    return y, s, mean, rstd


def check_bwd(b, dy, s, gamma, mean, rstd, skip, **kw):
    dx, dgamma, dbeta = b.swiglu_mlp_layer_norm_bwd(dy, s, gamma, mean, rstd, dskip=skip, **kw)
    M = s.shape[0]
    d, rs, mu = dy.double(), rstd.double()[:, None], mean.double()[:, None]
    w = torch.ones(s.shape[1], dtype=torch.float64, device="cuda") if gamma is None else gamma.double()
    xh, g = (s.double() - mu) * rs, d * w
    ref = rs * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    axh = rs * (s.double().abs() + mu.abs())
    scale = 200 * U * rs * (g.abs() + g.abs().mean(1, keepdim=True) + axh * (g.abs() * axh).mean(1, keepdim=True))
    if skip is not None:
        ref = ref + skip.double()
        scale = scale + U * ref.abs()
    within(dx, ref, scale, "dx")
    if dgamma is not None:
        within(dgamma, (d * xh).sum(0), (M + 100) * U * (d.abs() * axh).sum(0), "dgamma")
        within(dbeta, d.sum(0), (M + 100) * U * d.abs().sum(0), "dbeta")
    return dx, dgamma, dbeta


# widths: one column; fewer than a warp; a pack's tail; one warp; ragged multi-warp; the widest
# rows of each register form and one past it; rows and widths both odd
SHAPES = [(1, 1), (3, 7), (5, 8), (130, 100), (33, 256), (7, 257), (19, 1000), (4, 1023), (300, 1032), (9, 3584),
          (3, 8192), (5, 8193), (2, 8200), (3, 16384), (2, 16390), (3, 20001), (1300, 64),
          (2, 6144), (3, 6148), (2, 12288), (3, 12289), (700, 515), (5000, 24)]
TYPES = [(torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32), (torch.float16, torch.float16),
         (torch.float32, torch.float32)]


@pytest.mark.parametrize("types", TYPES, ids=str)
@pytest.mark.parametrize("M,D", SHAPES)
def test_forward_and_backward_match_fp64(b, M, D, types):
    t = draw(M, D, *types, seed=D)
    for r, skip in ((None, None), (t["r"], t["ds"])):
        _, s, mean, rstd = check_fwd(b, t, t["x"], r, t["gamma"], t["beta"])
        check_bwd(b, t["dy"], s, t["gamma"], mean, rstd, skip)


def test_no_parameters_and_parameters_alone(b):
    t = draw(37, 320, torch.bfloat16, torch.float32, 5)
    _, s, mean, rstd = check_fwd(b, t, t["x"], None, None, None)
    dx, dgamma, dbeta = check_bwd(b, t["dy"], s, None, mean, rstd, None, param_grads=False)
    assert dgamma is None and dbeta is None
    check_fwd(b, t, t["x"], t["r"], t["gamma"], None)
    check_fwd(b, t, t["x"], t["r"], None, t["beta"])
    check_bwd(b, t["dy"], s, None, mean, rstd, t["ds"])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D,pad,off", [(64, 8, 0), (64, 3, 0), (96, 2, 2), (264, 8, 1), (1000, 24, 8)])
def test_row_strides_and_unaligned_bases(b, dtype, D, pad, off):
    """Rows at a stride, bases that are aligned to the element only, columns past D untouched."""
    M = 21
    t = draw(M, D, dtype, torch.float32, 9)

    def wide(v=None):
        buf = torch.full((M, D + pad + off), 7.0, dtype=dtype, device="cuda")
        view = buf[:, off:off + D]
        if v is not None:
            view.copy_(v)
        return buf, view

    (_, x), (_, r), (_, dy), (_, ds) = (wide(t[k]) for k in ("x", "r", "dy", "ds"))
    (by, y), (bs, s), (bx, dx) = wide(), wide(), wide()
    _, _, mean, rstd = check_fwd(b, t, x, r, t["gamma"], t["beta"], y=y, s=s)
    check_bwd(b, dy, s, t["gamma"], mean, rstd, ds, dx=dx)
    for buf in (by, bs, bx):
        keep = torch.ones(buf.shape[1], dtype=torch.bool)
        keep[off:off + D] = False
        assert bool((buf[:, keep.cuda()] == 7.0).all())
    # the same values from contiguous tensors, bit for bit up to the order of the sums
    y2 = b.swiglu_mlp_layer_norm_fwd(t["x"], t["gamma"], t["beta"], EPS, residual=t["r"])[0]
    assert (y2.double() - y.double()).abs().max() <= 2 * UT[dtype] * y2.abs().max() + 1e-4


def test_large_mean_and_constant_rows(b):
    """A mean 1000 times the deviation keeps its precision (two passes); a constant row gives
    beta, and rstd = 1 / sqrt(eps)."""
    t = draw(16, 2048, torch.float32, torch.float32, 3)
    x = t["x"] * 1e-3 + 1.0
    check_fwd(b, t, x, None, t["gamma"], t["beta"])
    x = torch.full((4, 2048), 3.25, device="cuda")
    y, _, mean, rstd = b.swiglu_mlp_layer_norm_fwd(x, t["gamma"], t["beta"], EPS)
    assert bool((mean == 3.25).all()) and torch.equal(y, t["beta"].expand(4, -1))
    assert torch.allclose(rstd, torch.full_like(rstd, EPS ** -0.5), rtol=1e-6)


def test_non_finite_rows_stay_their_own(b):
    t = draw(9, 300, torch.bfloat16, torch.bfloat16, 4)
    x = t["x"].clone()
    x[2, 17], x[5, 0] = float("nan"), float("inf")
    y, _, mean, rstd = b.swiglu_mlp_layer_norm_fwd(x, t["gamma"], t["beta"], EPS)
    y0 = b.swiglu_mlp_layer_norm_fwd(t["x"], t["gamma"], t["beta"], EPS)[0]
    bad = torch.tensor([i in (2, 5) for i in range(9)], device="cuda")
    assert bool(y[bad].isnan().all()) and torch.equal(y[~bad], y0[~bad])
    assert bool(mean[2].isnan()) and bool(rstd[5].isnan())
    dx = b.swiglu_mlp_layer_norm_bwd(t["dy"], x, t["gamma"], mean, rstd)[0]
    assert bool(dx[bad].isnan().all()) and bool(dx[~bad].isfinite().all())


def test_no_rows(b):
    x = torch.empty(0, 96, dtype=torch.bfloat16, device="cuda")
    gamma = torch.ones(96, device="cuda")
    y, _, mean, rstd = b.swiglu_mlp_layer_norm_fwd(x, gamma, gamma, EPS)
    assert y.shape == (0, 96) and mean.shape == (0,)
    dgamma, dbeta = torch.full((96,), 5.0, device="cuda"), torch.full((96,), 5.0, device="cuda")
    b.swiglu_mlp_layer_norm_bwd(x, x, gamma, mean, rstd, dgamma=dgamma, dbeta=dbeta)
    assert not dgamma.any() and not dbeta.any()


def test_rows_past_32_bit_offsets(b):
    """A row stride that puts the last rows more than 2^31 elements from the first."""
    ld, M, D = 3 * 2 ** 28, 4, 40
    buf = torch.empty((M - 1) * ld + D, dtype=torch.bfloat16, device="cuda")
    t = draw(M, D, torch.bfloat16, torch.float32, 6)
    x = buf.as_strided((M, D), (ld, 1))
    x.copy_(t["x"])
    _, s, mean, rstd = check_fwd(b, t, x, None, t["gamma"], t["beta"])
    check_bwd(b, t["dy"], x, t["gamma"], mean, rstd, None)


def test_same_bits_every_run_and_on_another_stream(b):
    t = draw(1111, 776, torch.bfloat16, torch.float32, 8)
    _, s, mean, rstd = b.swiglu_mlp_layer_norm_fwd(t["x"], t["gamma"], t["beta"], EPS, residual=t["r"])
    first = b.swiglu_mlp_layer_norm_bwd(t["dy"], s, t["gamma"], mean, rstd, dskip=t["ds"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = b.swiglu_mlp_layer_norm_bwd(t["dy"], s, t["gamma"], mean, rstd, dskip=t["ds"])
    torch.cuda.current_stream().wait_stream(side)
    for p, q in zip(first, again):
        assert torch.equal(p, q)


def test_gradient_against_differences(b):
    """The kernel's gradient (fp32) against central differences of the fp64 formula along a
    random direction; the differences' own error is O(h^2) = 1e-8 of the loss's third
    derivative, the gradient's at most 200 u of its terms: 1e-4 covers both."""
    t = draw(6, 200, torch.float32, torch.float32, 12)
    _, s, mean, rstd = b.swiglu_mlp_layer_norm_fwd(t["x"], t["gamma"], t["beta"], EPS)
    dx, dgamma, dbeta = b.swiglu_mlp_layer_norm_bwd(t["dy"], s, t["gamma"], mean, rstd)
    g = torch.Generator(device="cuda").manual_seed(1)
    args = [t["x"].double(), t["gamma"].double(), t["beta"].double()]
    loss = lambda x, w, c: (fwd_ref(x, w, c)[0] * t["dy"].double()).sum()  # noqa: E731
    for i, grad in enumerate((dx, dgamma, dbeta)):
        v = torch.randn(args[i].shape, generator=g, device="cuda", dtype=torch.float64)
        plus, minus = list(args), list(args)
        plus[i], minus[i] = args[i] + 1e-4 * v, args[i] - 1e-4 * v
        want = (loss(*plus) - loss(*minus)) / 2e-4
        got = (grad.double() * v).sum()
        assert abs(got - want) <= 1e-4 * (grad.double() * v).abs().sum(), i


def test_autograd(b):
    """layer_norm's gradients through y and the residual stream, against fp64 autograd."""
    t = draw(2 * 9, 136, torch.float32, torch.float32, 14)
    shape = (2, 9, 136)
    leaves = [t["x"].reshape(shape), t["gamma"], t["beta"], t["r"].reshape(shape)]
    mine = [v.clone().requires_grad_() for v in leaves]
    ref = [v.double().requires_grad_() for v in leaves]
    y, s = b.layer_norm(mine[0], mine[1], mine[2], EPS, residual=mine[3])
    (y * t["dy"].reshape(shape) + s.sin()).sum().backward()
    s64 = ref[0] + ref[3]
    y64 = torch.nn.functional.layer_norm(s64, (136,), ref[1], ref[2], EPS)
    (y64 * t["dy"].reshape(shape).double() + s64.sin()).sum().backward()
    for p, q in zip(mine, ref):
        assert p.grad.shape == q.grad.shape
        assert (p.grad.double() - q.grad).norm() <= 1e-5 * q.grad.norm()
    # no residual, no bias, an expanded (zero-stride) incoming gradient
    x, w = leaves[0].clone().requires_grad_(), leaves[1].clone().requires_grad_()
    y, s = b.layer_norm(x, w)
    assert s is x
    y.sum().backward()
    x64, w64 = leaves[0].double().requires_grad_(), leaves[1].double().requires_grad_()
    torch.nn.functional.layer_norm(x64, (136,), w64, None, EPS).sum().backward()
    assert (w.grad.double() - w64.grad).norm() <= 1e-4 * w64.grad.norm()
    assert (x.grad.double() - x64.grad).abs().max() <= 1e-4

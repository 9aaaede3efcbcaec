"""GPU tests of the compiled calls of the short operators (csrc/ops/short_calls.cpp) against the ctypes
calls that binding.py makes where an output is the caller's, and of what both refuse."""
import pytest
import torch

from helpers import ensure_library

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def b():
    ensure_library()
    from bwd_gemm_epilogue_gb300 import binding
    binding.lib()
    return binding


def z(*shape, dtype=BF):
    g = torch.Generator().manual_seed(sum(shape))
    return torch.randn(*shape, generator=g).to(dtype).cuda()


@pytest.mark.parametrize("dtype,wdtype", [(BF, BF), (BF, F32), (HF, HF), (F32, F32)])
@pytest.mark.parametrize("params,residual", [(True, True), (True, False), (False, True)])
def test_layer_norm_both_ways(b, dtype, wdtype, params, residual):
    M, D = 37, 200
    x, r, dy = z(M, D + 8, dtype=dtype)[:, :D], z(M, D, dtype=dtype), z(M, 2 * D, dtype=dtype)[:, :D]
    r = r if residual else None
    gamma, beta = (z(D, dtype=wdtype), torch.nn.Parameter(z(D, dtype=wdtype))) if params else (None, None)
    got = b.swiglu_mlp_layer_norm_fwd(x, gamma, beta, 1e-5, residual=r)
    y = torch.empty_like(got[0])
    want = b.swiglu_mlp_layer_norm_fwd(x, gamma, beta, 1e-5, residual=r, y=y)
    assert want[0] is y and all(torch.equal(p, q) for p, q in zip(got, want))
    assert residual or got[1] is x
    assert not got[0].requires_grad and got[0].is_contiguous() and got[2].dtype == F32
    _, s, mean, rstd = got
    back = b.swiglu_mlp_layer_norm_bwd(dy, s, gamma, mean, rstd, dskip=r)
    dx = torch.empty_like(back[0])
    again = b.swiglu_mlp_layer_norm_bwd(dy, s, gamma, mean, rstd, dskip=r, dx=dx)
    assert again[0] is dx and all(torch.equal(p, q) for p, q in zip(back, again))
    assert back[1].dtype == (wdtype if params else dtype)


def test_clip_both_ways(b):
    grads = [z(1000), z(7, 9, dtype=F32), z(0), z(33, dtype=HF)]
    out = [torch.empty_like(g) for g in grads]
    norm, same = b.swiglu_mlp_clip_grads(grads, 0.5, out=out)
    want = torch.empty((), device="cuda")
    ref = [torch.empty_like(g) for g in grads]
    b.swiglu_mlp_clip_grads(grads, 0.5, out=ref, norm=want)
    assert torch.equal(norm, want) and torch.equal(b.swiglu_mlp_grad_norm(grads), want)
    assert all(torch.equal(p, q) for p, q in zip(same, ref))
    place = [g.clone() for g in grads]
    _, got = b.swiglu_mlp_clip_grads(tuple(place), 0.5)
    assert all(p is q for p, q in zip(got, place)) and all(torch.equal(p, q) for p, q in zip(place, ref))


def test_routed_moe_both_ways_on_another_stream(b):
    T, E, D, H, k = 9, 6, 128, 64, 3
    args = z(T, D), z(E, D, dtype=F32), z(E, 2 * H, D), z(E, D, H), k
    r = z(T, D)
    want = b.swiglu_moe_routed_fwd(*args, renormalize=False, residual=r, y=torch.empty(T, D, dtype=BF, device="cuda"))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = b.swiglu_moe_routed_fwd(*args, renormalize=False, residual=r)
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want)) and got[1].dtype == torch.int32


def test_refusals_are_the_same(b):
    x, w = z(4, 64), z(64)
    m = torch.zeros(4, device="cuda")
    W1, W2, Wr = z(6, 128, 64), z(6, 64, 64), z(6, 64)
    routed = b.swiglu_moe_routed_fwd
    cases = [
        (lambda: b.swiglu_mlp_layer_norm_fwd(x, w[:32]), ValueError),
        (lambda: b.swiglu_mlp_layer_norm_fwd(x, w.cpu()), ValueError),
        (lambda: b.swiglu_mlp_layer_norm_fwd(x.cpu()), ValueError),
        (lambda: b.swiglu_mlp_layer_norm_fwd(x.double()), TypeError),
        (lambda: b.swiglu_mlp_layer_norm_fwd(x, w.half()), TypeError),
        (lambda: b.swiglu_mlp_layer_norm_fwd(x.T), ValueError),
        (lambda: b.swiglu_mlp_layer_norm_fwd(x, residual=z(4, 32)), ValueError),
        (lambda: b.swiglu_mlp_layer_norm_fwd(x, eps=-1.0), b.SwigluError),
        (lambda: b.swiglu_mlp_layer_norm_bwd(x, x, w, m[:3], m), ValueError),
        (lambda: b.swiglu_mlp_layer_norm_bwd(x.float(), x, w, m, m), TypeError),
        (lambda: b.swiglu_mlp_clip_grads([x, w], 1.0, out=[w, x]), ValueError),
        (lambda: b.swiglu_mlp_clip_grads([x.T], 1.0), ValueError),
        (lambda: b.swiglu_mlp_clip_grads([x.long()], 1.0), TypeError),
        (lambda: b.swiglu_mlp_clip_grads([x], float("nan")), b.SwigluError),
        (lambda: routed(x, Wr, W1, z(6, 64, 32), 2), ValueError),
        (lambda: routed(x, Wr.half(), W1, W2, 2), TypeError),
        (lambda: routed(x, Wr, W1, W2, 7), b.SwigluError),
        (lambda: routed(x, Wr, W1, W2, 0), b.SwigluError),
        (lambda: routed(z(65, 64), Wr, W1, W2, 2), b.SwigluError),
    ]
    for i, (call, kind) in enumerate(cases):
        with pytest.raises(kind):
            call()
            pytest.fail(f"case {i} was not refused")
    assert b.swiglu_mlp_device_status() == 0

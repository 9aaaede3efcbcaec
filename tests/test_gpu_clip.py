"""GPU tests of the gradient clipping (swiglu_mlp_clip_grads, swiglu_mlp_grad_norm) against
fp64 torch.

Tolerances.  u = 2^-24.  A thread adds at most 17 fp32 squares of a chunk into each of two
sums, everything above that is fp64, so the sum's error is at most 20 u and the norm's 10 u,
plus its rounding to fp32: 12 u.  A clipped element carries the factor's error (11 u more), the
product's and the rounding to its type.
"""
import math

import pytest
import torch

from helpers import ensure_library

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
UT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: U}
TINY = {torch.bfloat16: 1e-38, torch.float16: 2.0 ** -24, torch.float32: 1e-38}
EPS = 1e-6
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def b():
    ensure_library()
    from bwd_gemm_epilogue_gb300 import binding
    binding.lib()
    return binding


def grads_of(shapes, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return [(std * torch.randn(n, generator=g)).to(d).cuda() for n, d in shapes]


def norm64(grads):
    return math.sqrt(sum(t.double().square().sum().item() for t in grads))


def check(b, grads, max_norm, out=None):
    before = [t.clone() for t in grads]
    want = norm64(before)
    factor = min(1.0, max_norm / (want + EPS))
    norm, got = b.swiglu_mlp_clip_grads(grads, max_norm, EPS, out=out)
    assert norm.dtype == F32 and norm.shape == ()
    assert abs(norm.item() - want) <= 12 * U * want
    for i, (p, q) in enumerate(zip(got, before)):
        assert p.dtype == q.dtype and p.shape == q.shape
        ref = q.double() * factor
        bound = ref.abs() * (UT[p.dtype] + 24 * U) + TINY[p.dtype]
        assert bool(((p.double() - ref).abs() <= bound).all()), i
        if out is not None:
            assert torch.equal(grads[i], q), "inputs are not written"
    assert abs(b.swiglu_mlp_grad_norm(before).item() - want) <= 12 * U * want
    return norm, got


LISTS = {
    "one element": [(1, F32)],
    "one bf16": [(5, BF)],
    "mixed types": [(1000, BF), (17, F32), (4097, HF), ((33, 65), F32), (1, BF)],
    "empty tensors": [(0, BF), (3, BF), (0, F32), ((0, 5), HF), (100, F32), (0, BF)],
    "only empty": [(0, BF), (0, F32)],
    "chunk edges": [(16384, BF), (16385, BF), (8191, F32), (8192, F32), (8193, F32), (32768, HF), (16383, HF)],
    "many chunks": [(3000001, BF), (1500003, F32)],
    "a few more than the small table": [(7 + i, [BF, F32, HF][i % 3]) for i in range(65)],
    "more than one launch": [(1 + i % 9, [BF, HF, F32][i % 3]) for i in range(1700)],
}


@pytest.mark.parametrize("name", list(LISTS))
@pytest.mark.parametrize("max_norm", [0.25, 1e9])
def test_matches_fp64(b, name, max_norm):
    grads = grads_of(LISTS[name], 3)
    check(b, grads, max_norm, out=[torch.empty_like(t) for t in grads])
    check(b, grads, max_norm)


@pytest.mark.parametrize("dtype", [BF, HF, F32])
def test_unaligned_views(b, dtype):
    """Views that start at any element of a buffer, outputs in step with them or not; what
    surrounds the views is not touched."""
    g = torch.Generator().manual_seed(5)
    buf = torch.randn(60000, generator=g).to(dtype).cuda()
    keep = buf.clone()
    views = [buf[1:1], buf[1:2], buf[3:9], buf[11:1029], buf[1030:35001], buf[35002:59995]]
    outbuf = torch.full((70000,), 9.0, dtype=dtype, device="cuda")
    out = [outbuf[s:s + v.numel()] for v, s in zip(views, (0, 8, 11, 27, 1101, 40000))]
    check(b, views, 0.5, out=out)
    assert bool((outbuf[59995 + 4998 + 1:] == 9.0).all()) and bool((outbuf[:8] == 9.0).all())
    check(b, views, 0.5)
    for i in (0, 2, 9, 10, 1029, 35001, 59995, 59999):
        assert buf[i] == keep[i]


def test_zero_gradients(b):
    grads = [torch.zeros(5000, dtype=BF, device="cuda"), torch.zeros(3, device="cuda")]
    norm, got = b.swiglu_mlp_clip_grads(grads, 1.0, EPS)
    assert norm.item() == 0.0 and not any(t.any() for t in got)
    norm, got = b.swiglu_mlp_clip_grads([t.fill_(2.0) for t in grads], 0.0, EPS)
    assert not any(t.any() for t in got), "max_norm 0 clips everything away"


def test_values_whose_squares_leave_fp32(b):
    """Finite bf16 and fp32 elements above 1.8e19: the norm is the fp64 one."""
    grads = grads_of([(40000, BF), (999, F32)], 7)
    grads[0][12345] = 3e30
    grads[1][5] = -2e25
    check(b, grads, 1.0, out=[torch.empty_like(t) for t in grads])


def test_non_finite_norm_follows_the_formulas(b):
    for bad in (float("inf"), float("-inf"), float("nan")):
        grads = grads_of([(40000, BF), (999, F32)], 8)
        grads[0][123] = bad
        norm, got = b.swiglu_mlp_clip_grads(grads, 1.0, EPS, out=[torch.empty_like(t) for t in grads])
        if math.isnan(bad):
            assert norm.isnan() and all(bool(t.isnan().all()) for t in got)
        else:
            assert norm.item() == math.inf
            assert bool(got[0][123].isnan()) and got[0].isnan().sum() == 1 and not got[1].any()


def test_same_bits_every_run_on_another_stream_and_in_a_graph(b):
    grads = grads_of([(300001, BF), (70001, F32), (9, HF)], 9, std=1e-3)
    out = [torch.empty_like(t) for t in grads]
    norm = torch.empty((), device="cuda")
    ws = torch.empty(b.swiglu_mlp_clip_grads_workspace_size(3), dtype=torch.uint8, device="cuda")
    b.swiglu_mlp_clip_grads(grads, 0.1, EPS, out=out, norm=norm, workspace=ws)
    want, want_norm = [t.clone() for t in out], norm.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            b.swiglu_mlp_clip_grads(grads, 0.1, EPS, out=out, norm=norm, workspace=ws)
        for t in out:
            t.zero_()
        graph.replay()
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(norm, want_norm) and all(torch.equal(p, q) for p, q in zip(out, want))

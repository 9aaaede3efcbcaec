"""GPU tests of the compiled calls of the operators of include/swiglu_tokens.h against the ctypes calls, which
binding.py makes where an output is the caller's or the module is missing, and of what both refuse."""
import pytest
import torch

from test_gpu_tokens import BF, F32, HF, SEED, b, case, rows_at  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF, HF, F32], ids=str)
def test_the_same_both_ways(b, monkeypatch, dtype):  # noqa: F811
    T, E, k, D = 23, 7, 3, 61
    ids, counts, pos, g = case(T, E, k, 0.2, 8)
    N = int(counts.sum())
    x, rows, res, dy = (rows_at(n, D, dtype, g, 64) for n in (T, N, T, T))
    logits, gates, dg = rows_at(T, E, dtype, g, 9), torch.rand(T, k, generator=g).cuda(), torch.randn(T, k, generator=g).cuda()
    step, add = torch.tensor(5, device="cuda"), rows_at(T, D, F32, g)
    mask = dict(p=0.5, seed=3, offset=4, step=step)
    big = dict(p=0.5, seed=SEED, offset=2 ** 64 - 1)       # past 63 bits

    def calls():
        out = [*b.swiglu_moe_gate_fwd(logits, k), *b.swiglu_moe_gate_fwd(logits, k, False),
               b.swiglu_moe_gate_bwd(logits, ids, gates, dg), b.swiglu_moe_gate_bwd(logits, ids, gates, dg, False),
               *b.swiglu_moe_sort(ids, E), b.swiglu_moe_dispatch_fwd(x, pos, N), b.swiglu_moe_dispatch_bwd(rows, pos),
               b.swiglu_moe_dispatch_bwd(rows, pos, add=add), b.swiglu_moe_dispatch_bwd(rows, pos, add=res),
               b.swiglu_moe_combine_fwd(rows, pos, gates), b.swiglu_moe_combine_fwd(rows, pos, gates, residual=res, **mask),
               b.swiglu_moe_combine_fwd(rows, pos, gates, **big), *b.swiglu_moe_combine_bwd(dy, rows, pos, gates),
               *b.swiglu_moe_combine_bwd(dy, rows, pos, gates, **mask), b.swiglu_mlp_dropout(x, **mask),
               b.swiglu_mlp_dropout(x, residual=res, **mask), b.swiglu_mlp_dropout(x, residual=res, **big)]
        spare = b.swiglu_moe_dispatch_fwd(x, pos)          # a row for every pair; those without one are unwritten
        return out + [spare[:N]]

    got = calls()
    assert b._short().moe_combine_fwd(rows, pos, gates, None, 0.5, 3, 4, step) is not None, "the compiled module is in use"
    monkeypatch.setattr(b, "_short_calls", b._NoShortCalls())
    want = calls()
    assert all(torch.equal(p, q) and p.dtype == q.dtype and p.is_contiguous() for p, q in zip(got, want))


def test_refusals_are_the_same(b):  # noqa: F811
    l, ids, q, x, rows = (torch.zeros(s, dtype=t, device="cuda") for s, t in
                          (((6, 9), BF), ((6, 3), torch.int32), ((6, 3), F32), ((6, 40), BF), ((11, 40), BF)))
    cases = [
        (lambda: b.swiglu_moe_gate_fwd(l.double(), 3), TypeError),
        (lambda: b.swiglu_moe_gate_fwd(l, 10), ValueError),
        (lambda: b.swiglu_moe_gate_fwd(torch.zeros(2, 1025, device="cuda"), 2), b.SwigluError),
        (lambda: b.swiglu_moe_gate_bwd(l, ids.long(), q, q), TypeError),
        (lambda: b.swiglu_moe_gate_bwd(l, ids, q.cpu(), q), ValueError),
        (lambda: b.swiglu_moe_sort(ids.long(), 4), TypeError),
        (lambda: b.swiglu_moe_sort(ids, 0), b.SwigluError),
        (lambda: b.swiglu_moe_sort(ids, 1025), b.SwigluError),
        (lambda: b.swiglu_moe_dispatch_fwd(x, ids[1:].contiguous()), ValueError),
        (lambda: b.swiglu_moe_dispatch_fwd(x, ids, -3), ValueError),
        (lambda: b.swiglu_moe_dispatch_bwd(rows, ids, add=x.half()), TypeError),
        (lambda: b.swiglu_moe_combine_fwd(rows, ids, q, p=1.5), b.SwigluError),
        (lambda: b.swiglu_moe_combine_fwd(rows, ids, q, residual=x[1:]), ValueError),
        (lambda: b.swiglu_moe_combine_fwd(rows.cpu(), ids, q), ValueError),
        (lambda: b.swiglu_moe_combine_bwd(x.float(), rows, ids, q), TypeError),
        (lambda: b.swiglu_mlp_dropout(x, 0.5, -1), ValueError),
        (lambda: b.swiglu_mlp_dropout(x, float("nan"), 1), b.SwigluError),
        (lambda: b.swiglu_mlp_dropout(x.t(), 0.5, 1), ValueError),
        (lambda: b.swiglu_mlp_dropout(x, 0.5, 1, step=torch.tensor(1)), ValueError),
    ]
    for i, (call, kind) in enumerate(cases):
        with pytest.raises(kind):
            call()
            pytest.fail(f"case {i} was not refused")
    assert b.swiglu_mlp_device_status() == 0

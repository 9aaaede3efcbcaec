"""GPU tests of the order of launches that come up while the kernel before them ends: what one call writes the
next one reads, however they are queued."""
import pytest
import torch

from test_gpu_moe_block import batch, params
from test_gpu_tokens import BF, F32, b  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,D", [(BF, 512), (F32, 61), (BF, 1021)])
def test_calls_in_a_row_see_what_the_call_before_wrote(b, dtype, D):  # noqa: F811
    """A chain of short calls over the same buffers, queued at once and one at a time."""
    g = torch.Generator(device="cuda").manual_seed(1)
    T, E, k, turns = 64, 8, 2, 40
    x0 = torch.randn(T, D, device="cuda", generator=g).to(dtype)
    logits0 = torch.randn(T, E, device="cuda", generator=g)

    def chain(wait):
        x, logits, rows = x0.clone(), logits0.clone(), torch.zeros(T * k, D, dtype=dtype, device="cuda")
        ids, pos = (torch.empty(T, k, dtype=torch.int32, device="cuda") for _ in range(2))
        gates, dgates = (torch.empty(T, k, device="cuda") for _ in range(2))
        counts = torch.empty(E, dtype=torch.int32, device="cuda")
        step = torch.zeros((), dtype=torch.int64, device="cuda")
        seen = []
        for i in range(turns):
            for call in (lambda: b.swiglu_moe_gate_fwd(logits, k, ids=ids, gates=gates),
                         lambda: b.swiglu_moe_sort(ids, E, counts=counts, pos=pos),
                         lambda: b.swiglu_moe_dispatch_fwd(x, pos, rows=rows),
                         lambda: b.swiglu_mlp_dropout(rows, 0.25, 3, offset=i, step=step, y=rows),
                         lambda: b.swiglu_moe_combine_fwd(rows, pos, gates, residual=x, y=x),
                         lambda: b.swiglu_moe_combine_bwd(x, rows, pos, gates, drows=rows.new_zeros(rows.shape), dgates=dgates),
                         lambda: b.swiglu_moe_gate_bwd(logits, ids, gates, dgates, dlogits=logits),
                         lambda: logits.add_(logits0).clamp_(-4, 4),
                         lambda: x.clamp_(-2, 2),
                         lambda: step.add_(1)):
                call()
                if wait:
                    torch.cuda.synchronize()
            seen.append((x.clone(), logits.clone(), pos.clone(), counts.clone()))
        return seen

    for got, want in zip(chain(False), chain(True)):
        assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_a_captured_fork_and_join(b):  # noqa: F811
    """Calls on two streams that wait for one another, captured into one graph."""
    x = torch.randn(300, 200, device="cuda").to(BF)
    main, side = torch.cuda.Stream(), torch.cuda.Stream()

    def calls():
        side.wait_stream(torch.cuda.current_stream())
        a = b.swiglu_mlp_dropout(x, 0.5, 1)
        with torch.cuda.stream(side):
            c = b.swiglu_mlp_dropout(x, 0.5, 2)
            side.wait_stream(main)
            c = b.swiglu_mlp_dropout(a, 0.25, 3, residual=c)
        a2 = b.swiglu_mlp_dropout(a, 0.5, 4)
        main.wait_stream(side)
        return b.swiglu_mlp_dropout(a2, 0.5, 5, residual=c)

    main.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(main):
        calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=main):
        out = calls()
    for turn in range(3):
        x.copy_(torch.randn(300, 200, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        a = b.swiglu_mlp_dropout(x, 0.5, 1)
        c = b.swiglu_mlp_dropout(a, 0.25, 3, residual=b.swiglu_mlp_dropout(x, 0.5, 2))
        assert torch.equal(out, b.swiglu_mlp_dropout(b.swiglu_mlp_dropout(a, 0.5, 4), 0.5, 5, residual=c))


def test_the_block_queued_at_once_and_call_by_call(b, monkeypatch):  # noqa: F811
    from bwd_gemm_epilogue_gb300.moe_block import PreNormMoE

    def train():
        block = PreNormMoE(*(p.clone() for p in params(6, 136, 72, 1)), top_k=2, dropout=0.1, seed=5)
        out = []
        for i in range(6):
            out += [block.forward(batch(90, 136, i)), block.backward(batch(90, 136, 50 + i)), block.step(0.1, 1.0)]
        return out + block.params

    want = train()
    for name in [n for n in vars(b) if n.startswith("swiglu_m") and n.endswith(("_fwd", "_bwd", "_sort", "_grads"))]:
        plain = getattr(b, name)
        monkeypatch.setattr(b, name, lambda *a, _f=plain, **k: (_f(*a, **k), torch.cuda.synchronize())[0])
    assert all(torch.equal(p, q) for p, q in zip(train(), want))

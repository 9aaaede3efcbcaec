"""GPU tests of the stack's dropout masks from call to call: in a captured graph, and in a run that is resumed."""
import pytest
import torch

from test_gpu_moe_block import batch
from test_gpu_tokens import b  # noqa: F401
from tokens_reference import keep_mask

pytestmark = pytest.mark.gpu
L, M, D, H, P, SEED = 3, 128, 128, 64, 0.5, 77


@pytest.fixture
def stack(b):  # noqa: F811
    from bwd_gemm_epilogue_gb300.stack import SwiGLUStack
    from bwd_gemm_epilogue_gb300 import workloads
    layers = [tuple(w.cuda() for w in workloads.make_weights(workloads.Shape(M, D, H, D), 5 + l)) for l in range(L)]
    return lambda: SwiGLUStack(layers, M, dropout=P, seed=SEED)


def results(stack, dy):
    """Outputs of every layer, dx and the weights' gradients."""
    dx, grads = stack.backward(dy)
    return [t.clone() for t in (*stack.acts[1:], dx, *(g for pair in grads for g in pair))]


def test_replays_have_masks_of_their_own(stack):
    st, eager = stack(), stack()
    x, dy = batch(M, D, 1), batch(M, D, 2)
    step = torch.zeros((), dtype=torch.int64, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        st.forward(x, step)
        st.backward(dy)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step += 1
        st.forward(x, step)
        out = results(st, dy)
    step.fill_(40)
    kept = []
    for i in (41, 42, 43):
        graph.replay()
        eager.forward(x, torch.tensor(i, device="cuda"))
        assert step.item() == i and all(torch.equal(p, q) for p, q in zip(out, results(eager, dy)))
        for l in range(L):
            mask, _ = keep_mask(M, D, P, SEED, (l << 48) + (1 << 47) + i)
            assert not out[l][~mask].any()
            kept.append(mask)
    for i, p in enumerate(kept):                           # independent: equal with chance 0.5
        for q in kept[:i]:
            assert abs((p == q).float().mean().item() - 0.5) < 6 * 0.5 / (M * D) ** 0.5


def test_a_captured_call_needs_a_step(stack):
    st = stack()
    x, dy = batch(M, D, 1), batch(M, D, 2)
    st.forward(x)
    before = results(st, dy)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dy + x
        for call in (lambda: st.forward(x), lambda: st.backward(dy)):
            with pytest.raises(ValueError, match="step"):
                call()
    st.calls = 0
    st.forward(x)
    assert all(torch.equal(p, q) for p, q in zip(before, results(st, dy)))
    st.dropout = 0.0                                       # nothing to repeat
    st.forward(x)
    st.backward(dy)
    torch.cuda.synchronize()
    with torch.cuda.graph(torch.cuda.CUDAGraph()):
        st.forward(x)
        st.backward(dy)


def test_a_resumed_run_goes_on_with_its_masks(stack):
    x, dy = batch(M, D, 1), batch(M, D, 2)
    a, c = stack(), stack()
    for _ in range(3):
        a.forward(x)
    c.calls = 2
    c.forward(x)
    assert c.calls == a.calls == 3
    assert all(torch.equal(p, q) for p, q in zip(results(a, dy), results(c, dy)))


def test_a_mask_is_the_same_in_both_directions(stack):
    """Whatever is set between them."""
    x, dy = batch(M, D, 1), batch(M, D, 2)
    a, c = stack(), stack()
    a.forward(x)
    c.forward(x)
    c.dropout, c.calls, c.seed = 0.25, 9, 1
    assert all(torch.equal(p, q) for p, q in zip(results(a, dy), results(c, dy)))

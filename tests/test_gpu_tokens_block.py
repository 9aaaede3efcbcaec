"""GPU tests of a token's way to its experts and back as it is used: through autograd, in the pre-norm MoE
block and in the stack of blocks with dropout."""
import pytest
import torch

from helpers import parity
from test_gpu_moe_block import batch, params, reference
from test_gpu_tokens import BF, F32, b, case, rows_at  # noqa: F401
from tokens_reference import keep_mask

pytestmark = pytest.mark.gpu


def close(got, want, what, rel=1e-5):
    """Norms, fp32 against fp64: sums of a few hundred products, each off by 2^-24 of itself."""
    d = (got.double() - want.double()).norm() / want.double().norm().clamp(min=1e-30)
    assert got.shape == want.shape and d <= rel, f"{what}: {d.item():.2e}"


@pytest.mark.parametrize("p", [0.0, 0.4])
@pytest.mark.parametrize("renormalize", [True, False])
def test_autograd_against_fp64(b, renormalize, p):  # noqa: F811
    """x -> gate, dispatch, a matrix for each expert, combine; the gradients of all leaves against fp64's."""
    lead, D, E, k = (5, 7), 24, 6, 3
    T = 35
    g = torch.Generator().manual_seed(2)
    leaf = lambda *s: torch.randn(*s, generator=g).cuda().requires_grad_()  # noqa: E731
    x, w, W, res = leaf(*lead, D), leaf(E, D), leaf(E, D, D), leaf(*lead, D)
    logits = x @ w.T
    ids, gates = b.moe_gate(logits, k, renormalize)
    assert ids.shape == (*lead, k) and not ids.requires_grad
    counts, pos = b.swiglu_moe_sort(ids, E)
    n = counts.tolist()
    rows = b.moe_dispatch(x, pos, sum(n))
    out = torch.cat([r @ W[e] for e, r in enumerate(rows.split(n))])
    y = b.moe_combine(out, pos, gates, res, p, 7, 8)
    up = torch.randn(*lead, D, generator=g).cuda()
    y.backward(up)

    x64, w64, W64, r64 = (t.detach().double().requires_grad_() for t in (x, w, W, res))
    prob = torch.softmax(x64 @ w64.T, -1)
    q = torch.gather(prob, -1, ids.long())
    q = q / q.sum(-1, keepdim=True) if renormalize else q
    branch = (torch.einsum("abd,abkde->abke", x64, W64[ids.long()]) * q[..., None]).sum(-2)
    if p:
        mask, f = keep_mask(T, D, p, 7, 8)
        branch = branch * (mask * f).view(*lead, D)
    y64 = r64 + branch
    y64.backward(up.double())
    close(y, y64, "y")
    for name, a, c in (("x", x, x64), ("w", w, w64), ("W", W, W64), ("residual", res, r64)):
        close(a.grad, c.grad, name)
    assert res.grad.data_ptr() != up.data_ptr()


def test_autograd_of_dropout(b):  # noqa: F811
    x, r = torch.randn(3, 4, 50, device="cuda", requires_grad=True), torch.randn(12, 50, device="cuda", requires_grad=True)
    step = torch.tensor(4, device="cuda")
    y = b.dropout(x, 0.3, 9, 2, step, r.view(3, 4, 50))
    y.sum().backward()
    mask, f = keep_mask(12, 50, 0.3, 9, 6)
    want = (mask * f).float()
    assert torch.equal(x.grad.view(12, 50), want) and torch.equal(r.grad, torch.ones_like(r))
    y = b.dropout(x, 0.3, 9, 2, step)
    step += 1
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


def test_a_second_derivative_is_refused(b):  # noqa: F811
    l = torch.randn(6, 5, device="cuda", requires_grad=True)
    _, gates = b.moe_gate(l, 2)
    (d,) = torch.autograd.grad(gates.square().sum(), l, create_graph=True)
    with pytest.raises(RuntimeError, match="no second derivative"):
        d.sum().backward()


def test_rows_without_a_pair_have_no_gradient(b):  # noqa: F811
    ids, counts, pos, g = case(9, 4, 2, 0.4, 3)
    x = torch.randn(9, 16, device="cuda", requires_grad=True)
    rows = b.moe_dispatch(x, pos)                          # 18 rows, some without a pair: zeros
    n = int(counts.sum())
    assert rows.shape == (18, 16) and not rows[n:].any()
    rows = rows.detach().requires_grad_()
    b.moe_combine(rows, pos, torch.rand(9, 2, device="cuda")).sum().backward()
    assert rows.grad[:n].any(1).all() and not rows.grad[n:].any()


@pytest.mark.parametrize("T,E,k", [(70, 6, 2), (33, 24, 20), (1, 5, 1)])
def test_block_with_dropout_against_fp64(b, T, E, k):  # noqa: F811
    """Bars as in test_gpu_moe_block; with dropout the branch's terms grow by 1 / 0.75 at most."""
    from bwd_gemm_epilogue_gb300.moe_block import PreNormMoE
    D, H, p = 136, 72, 0.25
    w = params(E, D, H, 1)
    x, dy = batch(T, D, 2), batch(T, D, 3)
    block = PreNormMoE(*w, top_k=k, dropout=p, seed=123)
    for call in range(2):
        y, dx = block.forward(x), None
        dx = block.backward(dy)
        leaves = [t.double().requires_grad_() for t in w]
        x64 = x.double().requires_grad_()
        mask, f = keep_mask(T, D, p, 123, call)
        y64 = x64 + (reference(leaves, x64, block._saved[4]) - x64) * (mask * f)
        y64.backward(dy.double())
        parity(y, y64.detach().cpu().numpy(), "y")
        for name, got, want in zip(("dx", "dgamma", "dbeta", "drouter", "dW1", "dW2"), [dx] + block.grads,
                                   [x64.grad] + [t.grad for t in leaves]):
            if T > 1 or name not in ("drouter",):          # one choice of one: its gate is 1 whatever the router
                parity(got, want.cpu().numpy(), name, rel_fro=1e-2, max_abs_frac=4e-2)
    assert block.calls == 2


def test_block_of_no_tokens(b):  # noqa: F811
    from bwd_gemm_epilogue_gb300.moe_block import PreNormMoE
    block = PreNormMoE(*params(4, 64, 32, 1), top_k=2)
    x = batch(0, 64, 1)
    assert block.forward(x).shape == (0, 64) and block.backward(x).shape == (0, 64)
    assert all(not g.any() for g in block.grads)


def test_stack_with_dropout(b):  # noqa: F811
    from bwd_gemm_epilogue_gb300.stack import SwiGLUStack
    from bwd_gemm_epilogue_gb300 import workloads
    L, M, D, H, p = 3, 200, 128, 192, 0.2
    layers = [tuple(w.cuda() for w in workloads.make_weights(workloads.Shape(M, D, H, D), 50 + l)) for l in range(L)]
    x, dy = batch(M, D, 2), batch(M, D, 3)
    stack = SwiGLUStack(layers, M, dropout=p, seed=31)
    for call in (1, 2):
        y = stack.forward(x).clone()
        dx, grads = stack.backward(dy)
        cur, saved = x, []
        for l, (W1, W2) in enumerate(layers):
            preact, out = b.swiglu_mlp_fwd(cur, W1, W2)
            mask, f = keep_mask(M, D, p, 31, call * L + l)
            saved.append((cur, preact, mask, f))
            cur = torch.where(mask, out.float() * f, 0).to(BF)
        assert torch.equal(y, cur)
        cur = dy
        for l in reversed(range(L)):
            inp, preact, mask, f = saved[l]
            cur, dW1, dW2 = b.swiglu_mlp_bwd(inp, *layers[l], preact, torch.where(mask, cur.float() * f, 0).to(BF))
            assert torch.equal(dW1, grads[l][0]) and torch.equal(dW2, grads[l][1])
        assert torch.equal(dx, cur)
    with pytest.raises(ValueError, match="dropout"):
        SwiGLUStack(layers, M, dropout=1.5)

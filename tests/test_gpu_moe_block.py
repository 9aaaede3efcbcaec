"""The pre-norm MoE block (moe_block.PreNormMoE): its training step against fp64 autograd, its
decode against its forward, and a few steps of training on one batch."""
import pytest
import torch

from helpers import ensure_library, parity

pytestmark = pytest.mark.gpu
bf = torch.bfloat16


@pytest.fixture(scope="module")
def Block():
    ensure_library()
    from bwd_gemm_epilogue_gb300.moe_block import PreNormMoE
    return PreNormMoE


def params(E, D, H, seed, router=torch.float32):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s, std=1.0: std * torch.randn(s, generator=g)  # noqa: E731
    return [(1 + 0.1 * n(D)).cuda(), (0.1 * n(D)).cuda(), n(E, D, std=2 * D ** -0.5).to(router).cuda(),
            n(E, 2 * H, D, std=D ** -0.5).to(bf).cuda(), n(E, D, H, std=H ** -0.5).to(bf).cuda()]


def batch(T, D, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(T, D, generator=g).to(bf).cuda()


def reference(p, x, ids):
    """fp64, with the choice of experts given."""
    gamma, beta, router, W1, W2 = p
    H = W2.shape[2]
    xn = torch.nn.functional.layer_norm(x, (x.shape[1],), gamma, beta, 1e-5)
    gates = torch.softmax(torch.gather(xn @ router.T, 1, ids), 1)
    y = x
    for j in range(ids.shape[1]):
        z = torch.einsum("td,thd->th", xn, W1[ids[:, j]])
        h = z[:, :H] * torch.nn.functional.silu(z[:, H:])
        y = y + gates[:, j:j + 1] * torch.einsum("th,tdh->td", h, W2[ids[:, j]])
    return y


def test_training_step_matches_fp64_autograd(Block):
    """Bar: the parity bar of the block (5e-3), twice that for gradients that pass the layer
    norm and the router as well (two more bf16 roundings on their way)."""
    T, E, D, H, k = 70, 6, 136, 72, 2
    p = params(E, D, H, 1)
    x, dy = batch(T, D, 2), batch(T, D, 3)
    block = Block(*p, top_k=k)
    y = block.forward(x)
    dx = block.backward(dy)
    leaves = [t.double().requires_grad_() for t in p]
    x64 = x.double().requires_grad_()
    y64 = reference(leaves, x64, block._saved[4])
    y64.backward(dy.double())
    parity(y, y64.detach().cpu().numpy(), "y")
    for name, got, want in zip(("dx", "dgamma", "dbeta", "drouter", "dW1", "dW2"), [dx] + block.grads,
                               [x64.grad] + [t.grad for t in leaves]):
        parity(got, want.cpu().numpy(), name, rel_fro=1e-2, max_abs_frac=4e-2)


@pytest.mark.parametrize("T", [1, 7, 64])
@pytest.mark.parametrize("router", [torch.float32, bf])
def test_decode_matches_forward(Block, T, router):
    block = Block(*params(12, 264, 136, 4, router), top_k=3)
    x = batch(T, 264, 5)
    y = block.decode(x)
    parity(y, block.forward(x).double().cpu().numpy(), "decode", rel_fro=1e-2, max_abs_frac=4e-2)


def test_steps_lower_the_loss_and_clip(Block):
    block = Block(*params(8, 128, 64, 6), top_k=2)
    x, target = batch(256, 128, 7), batch(256, 128, 8)
    losses, norms = [], []
    for _ in range(8):
        diff = block.forward(x).float() - target.float()
        losses.append(diff.square().mean().item())
        block.backward((2 * diff / diff.numel()).to(bf))
        norms.append(block.step(lr=4.0, max_norm=0.05).item())
        total = sum(g.double().square().sum() for g in block.grads).sqrt().item()
        assert total <= 0.05 * (1 + 2.0 ** -8)
    assert losses[-1] < losses[0] and min(norms) > 0


def test_shapes_are_checked(Block):
    p = params(4, 64, 32, 9)
    with pytest.raises(ValueError, match="shape mismatch"):
        Block(p[0][:32], *p[1:], top_k=2)
    with pytest.raises(ValueError, match="top_k"):
        Block(*p, top_k=5)

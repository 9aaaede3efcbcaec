"""GPU tests of the dropout masks of several pre-norm MoE blocks, and of a run that is resumed."""
import pytest
import torch

from test_gpu_moe_block import batch, params
from test_gpu_tokens import b  # noqa: F401
from tokens_reference import keep_mask

pytestmark = pytest.mark.gpu
T, E, D, H, P = 200, 4, 64, 32, 0.5


@pytest.fixture
def block(b):  # noqa: F811
    from bwd_gemm_epilogue_gb300.moe_block import PreNormMoE
    weights = params(E, D, H, 1)
    return lambda **kw: PreNormMoE(*weights, top_k=2, dropout=P, **kw)


def kept(block, x):
    """Which elements of the branch are kept.  One that is not leaves x as it is; one that is moves it."""
    return block.forward(x) != x


def alike(p, q):
    return (p == q).float().mean().item()


def test_blocks_of_one_seed_have_masks_of_their_own(block):
    x = batch(T, D, 2)
    masks = []
    for layer in (0, 1, 65535):
        bl = block(seed=9, layer=layer)
        for call in range(2):
            masks.append(kept(bl, x))
            want, _ = keep_mask(T, D, P, 9, (layer << 48) + call)
            assert not masks[-1][~want].any() and alike(masks[-1], want) > 0.95        # a few are lost in x's rounding
    for i, p in enumerate(masks):                          # independent: equal with chance 0.5
        for q in masks[:i]:
            assert abs(alike(p, q) - 0.5) < 0.1


def test_blocks_without_a_seed_have_masks_of_their_own(block):
    x = batch(T, D, 2)
    torch.manual_seed(3)
    first, second = block(), block()
    p, q = kept(first, x), kept(second, x)
    assert first.seed != second.seed and abs(alike(p, q) - 0.5) < 0.1
    torch.manual_seed(3)
    assert torch.equal(kept(block(), x), p) and torch.equal(kept(block(), x), q)


def test_stacks_without_a_seed_have_masks_of_their_own(b):  # noqa: F811
    from bwd_gemm_epilogue_gb300.stack import SwiGLUStack
    w = [torch.randn(s, device="cuda").bfloat16() for s in ((64, 64), (64, 32))]
    assert SwiGLUStack([w], 16, dropout=0.1).seed != SwiGLUStack([w], 16, dropout=0.1).seed


def test_no_seed_is_drawn_without_dropout(b):  # noqa: F811
    from bwd_gemm_epilogue_gb300.moe_block import PreNormMoE
    before = torch.get_rng_state()
    PreNormMoE(*params(E, D, H, 1), top_k=2)
    assert torch.equal(torch.get_rng_state(), before)


def test_dropout_that_is_set_later_has_a_seed_of_its_own(block):
    x = batch(T, D, 2)
    masks = []
    for _ in range(2):
        bl = block()
        bl.dropout, bl.seed = 0.0, None                    # as a block without dropout begins
        bl.forward(x)
        assert bl.seed is None
        bl.dropout = P
        masks.append(kept(bl, x))
    assert abs(alike(*masks) - 0.5) < 0.1


def test_a_resumed_run_goes_on_with_its_masks(block):
    x, dy = batch(T, D, 2), batch(T, D, 3)
    a, c = block(seed=1), block(seed=1)
    for _ in range(3):
        y = a.forward(x)
    c.calls = 2
    assert torch.equal(c.forward(x), y) and c.calls == 3
    assert torch.equal(a.backward(dy), c.backward(dy))


def test_layers_are_checked(block):
    for layer in (-1, 65536):
        with pytest.raises(ValueError, match="layer"):
            block(seed=1, layer=layer)

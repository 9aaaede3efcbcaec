"""GPU tests of the routed MoE layer's router where its dot products are shortest, so that the
CTAs of a token's cluster hand over their logits almost at once (tolerances: test_gpu_moe_routed.py)."""
import pytest
import torch

from test_gpu_moe_routed import b, check, draw  # noqa: F401

pytestmark = pytest.mark.gpu


# clusters of 1, 2, 4 and 8 CTAs; the largest E gives a warp 11 logits, E = 9 leaves warps without one
@pytest.mark.parametrize("E", [3, 9, 16, 17, 33, 64, 65, 682])
@pytest.mark.parametrize("T", [1, 64])
def test_short_dot_products(b, T, E):  # noqa: F811
    t = draw(T, E, 8, 8, 8, seed=E)
    _, ids, gates = check(b, t, 2, False, None)
    for _ in range(20):
        again = b.swiglu_moe_routed_fwd(t["x"], t["Wr"], t["W1"], t["W2"], 2, renormalize=False)
        assert torch.equal(again[1], ids) and torch.equal(again[2], gates)

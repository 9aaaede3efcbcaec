"""GPU tests of the routed MoE layer where chunks of several experts' tokens, every number of 8-token
tiles and every split of the units occur (tolerances: test_gpu_moe_routed.py)."""
import pytest
import torch

from test_gpu_moe_routed import b, check, draw  # noqa: F401

pytestmark = pytest.mark.gpu

# (T, E, D, H, Dout, k): experts of one or a few groups of 8 hidden units, so that a chunk holds many
# of them; 5 to 64 tokens an expert; rows kept in shared memory and not; few units of wide rows
CASES = [(64, 40, 264, 8, 64, 7), (64, 120, 328, 16, 72, 3), (48, 30, 2056, 24, 48, 2), (64, 8, 520, 72, 136, 2),
         (64, 3, 520, 136, 136, 1), (64, 2, 264, 264, 264, 1), (50, 4, 1096, 40, 520, 2), (33, 12, 776, 1000, 264, 5),
         (1, 2, 4104, 24, 64, 1), (2, 3, 2048, 8, 16, 2), (4, 64, 1032, 248, 1032, 8), (8, 32, 512, 1024, 512, 2),
         (16, 6, 4096, 104, 2056, 6)]


@pytest.mark.parametrize("T,E,D,H,Dout,k", CASES)
def test_matches_fp64(b, T, E, D, H, Dout, k):  # noqa: F811
    t = draw(T, E, D, H, Dout, seed=T + 2 * E + D)
    check(b, t, k, True, t["r"])


@pytest.mark.parametrize("T,H", [(64, 8), (61, 40), (24, 200)])
def test_uneven_experts(b, T, H):  # noqa: F811
    """A router that sends most tokens to a few experts: 1 to 64 tokens of one, next to each other."""
    t = draw(T, 24, 520, H, 136, seed=T)
    t["Wr"][:4] += 0.5 * t["x"][:1] / 520 ** 0.5
    t["x"][: T // 2] += t["x"][:1].clone()
    _, ids, _ = check(b, t, 3, True, None)
    counts = torch.bincount(ids.flatten().long(), minlength=24)
    assert counts.max() >= T // 3 and counts[counts > 0].min() <= 8

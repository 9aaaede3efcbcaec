"""GPU tests of the gradient clipping's outputs side by side, and of overlapping ones, which are refused
(one gradient listed twice would be scaled twice, or once, as its CTAs happen to run)."""
import pytest
import torch

from test_gpu_clip import BF, F32, b, check  # noqa: F401

pytestmark = pytest.mark.gpu


def test_neighbours_inputs_read_twice_and_empty_tensors(b):  # noqa: F811
    buf = torch.randn(100000, generator=torch.Generator().manual_seed(1)).cuda()
    cuts = [0, 1, 1, 5, 4099, 4099, 50001, 100000]
    views = [buf[p:q] for p, q in zip(cuts, cuts[1:])]
    check(b, views, 0.5, out=[torch.empty_like(v) for v in views])
    check(b, views, 0.5)
    same = [buf, buf, buf[7:99]]                             # read, not written
    check(b, same, 0.5, out=[torch.empty_like(v) for v in same])
    assert b.swiglu_mlp_grad_norm([buf, buf]).isfinite()


def test_overlaps_are_refused_and_nothing_is_written(b):  # noqa: F811
    for many in (0, 80):
        g, h = (torch.randn(5000, generator=torch.Generator().manual_seed(i)).cuda() for i in (2, 3))
        more = [torch.ones(9, dtype=BF, device="cuda") for _ in range(many)]
        keep = [t.clone() for t in (g, h)]
        for grads, out in [([g, h, g], None), ([g, g[10:20]], None), ([g, h], [h, g]), ([g[1:]], [g[:-1]]),
                           ([g, h], [torch.empty_like(g)] * 2)]:
            with pytest.raises(b.SwigluError, match="overlap"):
                b.swiglu_mlp_clip_grads(grads + more, 0.1, out=None if out is None else out + more)
        assert all(torch.equal(p, q) for p, q in zip((g, h), keep)) and all(bool((t == 1).all()) for t in more)

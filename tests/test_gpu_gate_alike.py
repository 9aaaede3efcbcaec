"""GPU tests of the gate's choice among logits a few units of the last place apart, where one lane of a token
has most of them: falling logit, ties to the lowest index."""
import pytest
import torch

from test_gpu_tokens import F32, b  # noqa: F401

pytestmark = pytest.mark.gpu
STEP = 2.0 ** -23


def check(b, l, k):  # noqa: F811
    want = torch.sort(l.double(), dim=1, descending=True, stable=True)[1][:, :k]
    for renormalize in (True, False):
        ids, _ = b.swiglu_moe_gate_fwd(l, k, renormalize)
        wrong = (ids.long() != want).any(1).nonzero().flatten().tolist()
        assert not wrong, f"{len(wrong)} rows, first {wrong[0]}: {ids[wrong[0]].tolist()}, not {want[wrong[0]].tolist()}"


@pytest.mark.parametrize("E", [80, 100, 128])
@pytest.mark.parametrize("k", [7, 8])
def test_equal_logits_past_the_words_a_lane_keeps(b, E, k):  # noqa: F811
    """k - 1 experts of one lane are chosen for sure, and two more of it end its nine words; of two equal
    logits that follow, the first is that lane's tenth expert or another lane's."""
    rows = []
    for lane in range(8):
        own = list(range(lane, E, 8))
        for first in (own[-1], own[-1] - 1 if lane else own[-1] - 7):
            l = torch.full((E,), -5.0)
            l[own[:k - 1]] = 1 + 10 * STEP
            l[own[k - 1:9]] = 1.0
            l[first] = 1 + 5 * STEP
            l[E - 1 if first != E - 1 else E - 2] = 1 + 5 * STEP
            rows.append(l)
    check(b, torch.stack(rows).to(F32).cuda(), k)


@pytest.mark.parametrize("E", [65, 80, 100, 128])
def test_few_steps_in_one_lane(b, E):  # noqa: F811
    """One lane's experts and a few others at one of four values, all else far below; each row four times, as a
    warp has four tokens and chooses anew for all of them where it has to for one."""
    g = torch.Generator().manual_seed(E)
    T = 1 << 16
    lane = torch.randint(0, 8, (T, 1), generator=g)
    near = (torch.arange(E) % 8 == lane) | (torch.rand(T, E, generator=g) < 0.03)
    l = torch.where(near, 1 + torch.randint(0, 4, (T, E), generator=g) * STEP, -5.0).to(F32).repeat_interleave(4, 0).cuda()
    for k in (6, 7, 8):
        check(b, l, k)

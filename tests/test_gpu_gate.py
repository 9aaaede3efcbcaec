"""GPU tests of the gate (swiglu_moe_gate_fwd / _bwd) against plain forms in fp64.

Tolerances, with u = 2^-24.  A gate is e^(l - top) over a sum of such: the difference is off by u of
itself, which moves e^(l - top) by u |l - top| of it, expf by 2 ulp (4 u); the sum has up to 32 terms
and 5 shuffles (or k terms) of the same errors after each other, the division is off by u.  So a gate is
off by at most (2 span + 60) u of itself, span the largest |l - top| of its row that still counts
(terms below e^-30 of the sum move it by less than u all together).  A gradient q (g - s), with s off by (k + 60) u of
its terms, is off by (2 span + k + 130) u of q (|g| + sum q |g|).
"""
import math

import pytest
import torch

from tokens_reference import U, gate, within
from test_gpu_tokens import BF, F32, HF, b  # noqa: F401

pytestmark = pytest.mark.gpu
SHAPES = [(1, 1, 1), (1, 64, 8), (7, 2, 2), (64, 8, 2), (33, 33, 5), (130, 61, 7), (19, 128, 8), (5, 200, 16), (9, 512, 33),
          (3, 1000, 40), (2, 1024, 1024), (4099, 40, 6)]


def draw(T, E, dtype, seed, off=0.0, ld=None):
    g = torch.Generator().manual_seed(seed)
    l = (2 * torch.randn(T, E, generator=g)).to(dtype)
    l[torch.rand(T, E, generator=g) < off] = -math.inf
    l[torch.rand(T, generator=g) < off / 2] = -math.inf
    buf = torch.full((T, E if ld is None else ld), math.nan, dtype=dtype, device="cuda")
    buf[:, :E] = l.cuda()
    return buf[:, :E], g


def span(l):
    d = l.double()
    top = d.max(1, keepdim=True).values
    d = (top - d).nan_to_num(nan=0.0, posinf=0.0)
    return d.clamp(max=200).max(1, keepdim=True).values


def check(b, l, k, renormalize, g):  # noqa: F811
    ids, gates = b.swiglu_moe_gate_fwd(l, k, renormalize)
    want_ids, want, p = gate(l, k, renormalize)
    assert ids.dtype == torch.int32 and torch.equal(ids.long(), want_ids)
    within(gates, want, (2 * span(l) + 60) * U * want.abs(), "gates")
    dg = torch.randn(l.shape[0], k, generator=g).cuda()
    here = ids >= 0
    q, d = gates.double(), dg.double()
    dg = dg.masked_fill(~here, math.nan)                   # not read
    got = b.swiglu_moe_gate_bwd(l, ids, gates.masked_fill(~here, math.nan), dg, renormalize)
    q = torch.where(here, q, 0.0)
    s, mag = (q * d).sum(1, keepdim=True), (q * d).abs().sum(1, keepdim=True)
    slot = torch.where(here, want_ids, l.shape[1])

    def spread(v):
        return torch.zeros(l.shape[0], l.shape[1] + 1, dtype=torch.float64, device="cuda").scatter_add(1, slot, v)[:, :-1]

    if renormalize:
        ref, scale = spread(q * (d - s)), spread(q * (d.abs() + mag))
    else:
        ref, scale = p * (spread(torch.where(here, d, 0.0)) - s), p * (spread(torch.where(here, d, 0.0).abs()) + mag)
    within(got, ref, (2 * span(l) + k + 130) * U * scale, "dlogits")
    return ids, gates, got


@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("dtype", [BF, HF, F32], ids=str)
@pytest.mark.parametrize("T,E,k", SHAPES)
def test_matches_fp64(b, T, E, k, dtype, renormalize):  # noqa: F811
    for off, ld in ((0.0, None), (0.3, E + 3)):
        l, g = draw(T, E, dtype, T + E, off, ld)
        check(b, l, k, renormalize, g)


def test_no_tokens(b):  # noqa: F811
    l = torch.empty(0, 8, device="cuda")
    ids, gates = b.swiglu_moe_gate_fwd(l, 2)
    assert ids.shape == gates.shape == (0, 2) and b.swiglu_moe_gate_bwd(l, ids, gates, gates).shape == (0, 8)


def test_ties_go_to_the_lowest_index(b):  # noqa: F811
    l = torch.zeros(3, 70, device="cuda")
    l[1, ::2] = 1.0
    l[2] = -0.0
    l[2, 5] = 0.0                                          # -0 is 0
    ids, gates = b.swiglu_moe_gate_fwd(l, 4)
    assert ids.tolist() == [[0, 1, 2, 3], [0, 2, 4, 6], [0, 1, 2, 3]] and torch.equal(gates, torch.full_like(gates, 0.25))


@pytest.mark.parametrize("E", [7, 13, 30, 60, 100, 250, 300, 1000])
def test_logits_that_differ_in_their_last_bits(b, E):  # noqa: F811
    """Around +1 and -1, in steps of one to a few units of the last place, some equal; and far apart
    but for two that end the chosen and begin the rest."""
    g = torch.Generator().manual_seed(E)
    T = 64
    steps = torch.randint(0, 2 * E, (T, E), generator=g)
    l = (1 + steps.double() * 2.0 ** -23).float()
    l[::2] = -l[::2]
    l[40:] = torch.randn(T - 40, E, generator=g)
    k = min(E - 1, 6)
    top = torch.sort(l[50:], dim=1, descending=True)
    l[50:].scatter_(1, top[1][:, k:k + 1], torch.nextafter(top[0][:, k - 1:k], torch.tensor(-9e9)))
    l = l.cuda()
    for renormalize in (True, False):
        for n in (1, 2, k, min(E, 9)):
            check(b, l, n, renormalize, g)


@pytest.mark.parametrize("E", [9, 16, 40, 128, 200, 512, 1024])
def test_many_logits_alike(b, E):  # noqa: F811
    """All equal (a router that starts at zero); two values a unit of the last place apart, a few of either,
    or one after all that are equal; a run of neighbours in one lane's experts; the same, some off."""
    g = torch.Generator().manual_seed(E)
    up = torch.nextafter(torch.ones(()), torch.tensor(2.0))
    l = torch.ones(96, E)
    l[1] = 0
    for i in range(2, 40):
        l[i, torch.randperm(E, generator=g)[:1 + i % 7]] = up
    l[40:50] = torch.where(torch.rand(10, E, generator=g) < 0.5, up, torch.ones(()))
    for i in range(50, 60):
        l[i, E - 1 - (i - 50) % E] = up                     # the last ones in order
        l[i, : (i - 50) % E] = -1.0
    for i in range(60, 76):                                # every G-th expert, which one lane has
        l[i, (i % 8)::8 if i < 68 else 16] += torch.randperm(len(l[i, (i % 8)::8 if i < 68 else 16]), generator=g) * 2.0 ** -23
    l[76:86] = 1 + torch.randint(0, 3, (10, E), generator=g) * 2.0 ** -23
    l[86:] = torch.where(torch.rand(10, E, generator=g) < 0.3, -math.inf, l[76:86])
    l = l.cuda()
    for renormalize in (True, False):
        for n in (1, 3, min(8, E), min(9, E), min(16, E), min(32, E)):
            check(b, l, n, renormalize, g)


@pytest.mark.parametrize("dtype", [BF, HF, F32], ids=str)
def test_lowest_values_count_as_values(b, dtype):  # noqa: F811
    low = torch.finfo(dtype).min
    l = torch.full((2, 6), low, dtype=dtype, device="cuda")
    l[1, 3] = 1.0
    ids, gates = b.swiglu_moe_gate_fwd(l, 2)
    assert ids.tolist() == [[0, 1], [3, 0]] and gates.tolist() == [[0.5, 0.5], [1.0, 0.0]]
    assert b.swiglu_moe_gate_bwd(l, ids, gates, torch.ones_like(gates), False).isfinite().all()


def test_infinite_and_nan_logits(b):  # noqa: F811
    inf, nan = math.inf, math.nan
    l = torch.tensor([[0.0, inf, 1.0, inf], [0.0, nan, 1.0, -1.0], [nan, nan, -inf, -inf], [-inf, -inf, -inf, -inf], [-inf, 2.0, -inf, -inf]],
                     device="cuda")
    for renormalize in (True, False):
        ids, gates = b.swiglu_moe_gate_fwd(l, 3, renormalize)
        assert ids.tolist() == [[1, 3, 2], [2, 0, 3], [0, 1, -1], [-1, -1, -1], [1, -1, -1]]
        assert gates[:2].isnan().all() and gates[2, :2].isnan().all()
        assert gates[2, 2] == 0 and not gates[3].any() and gates[4].tolist() == [1, 0, 0]
        d = b.swiglu_moe_gate_bwd(l, ids, gates, torch.ones_like(gates), renormalize)
        assert not d[3:].any()


@pytest.mark.parametrize("E", [6, 40, 128, 300])
def test_nan_of_any_sign_and_payload(b, E):  # noqa: F811
    """A NaN ranks lowest and makes its token's gates NaN, and no other token's."""
    for bits in (0x7fc00000, 0xffc00000, 0x7f800001, 0xff800001, 0x7fffffff, 0xffffffff):
        for dtype, shift in ((F32, 0), (BF, 16)):
            l = torch.randn(32, E, device="cuda").to(dtype)
            raw = (bits >> shift) | (1 if shift and not bits & 0x7f0000 else 0)
            ints, width = (torch.int32, 32) if shift == 0 else (torch.int16, 16)
            l[5, 2] = torch.tensor([raw - (1 << width) if raw >> (width - 1) else raw], dtype=ints).view(dtype).cuda()[0]
            assert l.isnan().sum() == 1
            for renormalize in (True, False):
                ids, gates = b.swiglu_moe_gate_fwd(l, 3, renormalize)
                want_ids, want, _ = gate(l, 3, renormalize)
                assert torch.equal(ids.long(), want_ids) and torch.equal(gates.isnan(), want.isnan())
                assert gates[5].isnan().all() and not gates[torch.arange(32) != 5].isnan().any()


def test_an_index_twice_and_indices_that_are_none(b):  # noqa: F811
    """The gradient takes any ids: shares of one index add up."""
    l = torch.randn(1, 5, device="cuda")
    ids = torch.tensor([[3, 3, 9, -4]], dtype=torch.int32, device="cuda")
    q = torch.tensor([[0.25, 0.5, math.nan, math.inf]], device="cuda")
    g = torch.tensor([[1.0, -2.0, math.nan, 1.0]], device="cuda")
    s = 0.25 - 1.0
    d = b.swiglu_moe_gate_bwd(l, ids, q, g)
    want = torch.zeros(1, 5, dtype=torch.float64, device="cuda")
    want[0, 3] = 0.25 * (1 - s) + 0.5 * (-2 - s)
    within(d, want, 8 * U * torch.full_like(want, 3.0), "dlogits")
    d = b.swiglu_moe_gate_bwd(l, ids, q, g, False)
    p = torch.softmax(l.double(), 1)
    up = torch.zeros_like(p)
    up[0, 3] = 1 - 2
    within(d, p * (up - s), 200 * U * 3 * p, "dlogits of all")


def test_in_place_and_rows_at_a_stride(b):  # noqa: F811
    l, g = draw(45, 24, BF, 3, 0.1)
    for renormalize in (True, False):
        ids, gates = b.swiglu_moe_gate_fwd(l, 3, renormalize)
        dg = torch.randn(45, 3, generator=g).cuda()
        want = b.swiglu_moe_gate_bwd(l, ids, gates, dg, renormalize)
        wide = torch.full((45, 40), 7.0, dtype=BF, device="cuda")
        b.swiglu_moe_gate_bwd(l, ids, gates, dg, renormalize, dlogits=wide[:, 4:28])
        assert torch.equal(wide[:, 4:28], want) and bool((wide[:, :4] == 7).all()) and bool((wide[:, 28:] == 7).all())
        place = l.clone()
        assert b.swiglu_moe_gate_bwd(place, ids, gates, dg, renormalize, dlogits=place) is place and torch.equal(place, want)


@pytest.mark.parametrize("renormalize", [True, False])
def test_gradient_matches_differences(b, renormalize):  # noqa: F811
    """<dlogits, v> against (L(l + h v) - L(l - h v)) / 2h, L = <gates, w>, h = 2^-6.  The gates are off
    by less than 130 u = 8e-6 of themselves and sum to 1 at most, so the quotient is off by 8e-6 / h = 5e-4
    of |w|; the third derivative of a softmax along v is at most 8 max |v|^3 |w|: h^2 / 6 of that."""
    T, E, k, h = 40, 12, 3, 2.0 ** -6
    g = torch.Generator().manual_seed(1)
    l = torch.randn(T, E, generator=g).cuda()
    order = torch.sort(l, dim=1, descending=True)[0]
    far = (order[:, k - 1] - order[:, k]) > 0.2            # the choice is the same on both sides
    v = torch.rand(T, E, generator=g).cuda() * 2 - 1
    w = torch.rand(T, k, generator=g).cuda() * 2 - 1
    ids, gates = b.swiglu_moe_gate_fwd(l, k, renormalize)
    d = b.swiglu_moe_gate_bwd(l, ids, gates, w, renormalize)

    def loss(x):
        i, q = b.swiglu_moe_gate_fwd(x.contiguous(), k, renormalize)
        dense = torch.zeros(T, E, dtype=torch.float64, device="cuda").scatter_(1, i.long(), q.double())
        return (torch.gather(dense, 1, ids.long()) * w.double()).sum(1)

    diff = (loss(l + h * v) - loss(l - h * v)) / (2 * h)
    got = (d.double() * v.double()).sum(1)
    assert int(far.sum()) > 10
    assert bool(((diff - got).abs()[far] <= 5e-4 * 1.1 + 8 * h * h / 6).all())

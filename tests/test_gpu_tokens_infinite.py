"""GPU tests of the operators of include/swiglu_tokens.h where values are infinite or come to be: the result has the
infinity of its formula there, with its sign, NaN where that has NaN, and all else within the usual bounds."""
import math

import pytest
import torch

from test_gpu_tokens import BF, F32, HF, b, case, rows_at  # noqa: F401
from tokens_reference import U, dropped, picked, within

pytestmark = pytest.mark.gpu
T, E, K, SEED = 40, 8, 3, 21


def strictly_within(got, ref, scale, what):
    """within, and where ref is infinite, got is the same."""
    inf = ref.isinf()
    assert int(inf.sum()) > 0, f"{what}: no infinite value to look at"
    assert torch.equal(got.double()[inf], ref[inf]), f"{what}: infinities"
    assert not got[~inf].isinf().any(), f"{what}: infinite where the formula is not"
    within(got.masked_fill(inf, 0), ref.masked_fill(inf, 0), scale.masked_fill(inf, 0).nan_to_num(0, 0, 0), what)


def with_infinities(t, g, share=0.03):
    at = torch.rand(t.shape, generator=g).cuda()
    t[at < share] = math.inf
    t[at > 1 - share] = -math.inf
    return t


@pytest.mark.parametrize("dtype", [BF, HF, F32], ids=str)
@pytest.mark.parametrize("D", [64, 61])
def test_infinite_rows(b, D, dtype):  # noqa: F811
    """The sums have an infinity where one addend has one, NaN where two of them cancel."""
    ids, counts, pos, g = case(T, E, K, 0.2, 7)
    rows = with_infinities(rows_at(int(counts.sum()), D, dtype, g), g)
    res = with_infinities(rows_at(T, D, dtype, g), g)
    gates = torch.rand(T, K, generator=g).cuda() + 0.01
    r64, _ = picked(rows, pos)
    w = torch.where(pos >= 0, gates, 0.0).double()[:, :, None]
    terms = torch.where((pos >= 0)[:, :, None], r64 * w, 0.0)
    strictly_within(b.swiglu_moe_dispatch_bwd(rows, pos, add=res), r64.sum(1) + res.double(),
                    (K + 4) * U * (r64.abs().sum(1) + res.double().abs()), "dispatch's gradient")
    for p in (0.0, 0.5):
        ref, mag = dropped(terms.sum(1), p, SEED, 0), dropped(terms.abs().sum(1), p, SEED, 0)
        strictly_within(b.swiglu_moe_combine_fwd(rows, pos, gates, residual=res, p=p, seed=SEED), ref + res.double(),
                        (K + 4) * U * (mag + res.double().abs()), f"combine, p {p}")
        strictly_within(b.swiglu_moe_combine_fwd(rows, pos, gates, p=p, seed=SEED), ref, (K + 4) * U * mag, f"combine alone, p {p}")
        x64 = dropped(res.double(), p, SEED, 0)
        strictly_within(b.swiglu_mlp_dropout(res, p, SEED), x64, 3 * U * x64.abs(), f"dropout, p {p}")


@pytest.mark.parametrize("dtype", [BF, HF, F32], ids=str)
@pytest.mark.parametrize("D", [64, 61])
@pytest.mark.parametrize("p", [0.0, 0.5])
def test_infinite_gradients(b, D, dtype, p):  # noqa: F811
    ids, counts, pos, g = case(T, E, K, 0.2, 8)
    n = int(counts.sum())
    rows, dy = rows_at(n, D, dtype, g), with_infinities(rows_at(T, D, dtype, g), g, 0.004)
    gates = torch.rand(T, K, generator=g).cuda() + 0.01
    drows, dgates = b.swiglu_moe_combine_bwd(dy, rows, pos, gates, p=p, seed=SEED, drows=torch.zeros(n, D, dtype=dtype, device="cuda"))
    e = dropped(dy.double(), p, SEED, 0)
    r64, here = picked(rows, pos)
    t, j = torch.nonzero(here, as_tuple=True)
    want = torch.zeros(n, D, dtype=torch.float64, device="cuda")
    want[pos[t, j].long()] = e[t] * gates.double()[t, j, None]
    strictly_within(drows, want, 3 * U * want.abs(), "drows")
    terms = torch.where(here[:, :, None], e[:, None] * r64, 0.0)
    strictly_within(dgates, terms.sum(2), (D / 64 + 40) * U * terms.abs().sum(2), "dgates")


def test_fp16_sums_past_its_range(b):  # noqa: F811
    """Finite addends whose sum rounds to infinity, and one below the border that does not: 65520 is half
    way between the largest fp16 value and the next step."""
    rows = torch.tensor([[60000.0, -60000.0, 65504.0, 65504.0]] * 2, device="cuda").half()
    add = torch.tensor([[0.0, 0.0, -65504.0, -65504.0 + 15.0]], device="cuda")
    pos = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda")
    got = b.swiglu_moe_dispatch_bwd(rows, pos, add=add)
    assert got.tolist() == [[math.inf, -math.inf, 65504.0, 65504.0]]
    add[0, 3] += 1.0                                       # 65504 + 16: the tie goes to the even one, infinity
    assert b.swiglu_moe_dispatch_bwd(rows, pos, add=add).tolist() == [[math.inf, -math.inf, 65504.0, math.inf]]

"""GPU tests of a token's way to its experts and back and of dropout (include/swiglu_tokens.h) against
plain forms in fp64.

Tolerances, with u = 2^-24, before the one rounding of an output to its type: a sum over k choices
with the gates, dropout's factor and the residual takes k + 3 roundings at most, (k + 4) u of its terms'
magnitudes.  A dgate sums D products: at most D / 64 + 40 of them and of partial sums come one after the
other (256 threads with packs of 4 or more in two chains, 5 shuffles, 8 warps).  drows: three products.
"""
import pytest
import torch

from helpers import ensure_library
from tokens_reference import U, dropped, keep_mask, picked, sort, within

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
SEED = 0xfedcba9876543210


@pytest.fixture(scope="module")
def b():
    ensure_library()
    from bwd_gemm_epilogue_gb300 import binding
    binding.lib()
    return binding


def rows_at(M, D, dtype, g, ld=None, start=0, pad=float("nan")):
    """[M, D] normal values whose rows are `ld` elements apart, the first at element `start`; all else NaN."""
    ld = D if ld is None else ld
    buf = torch.full((start + M * ld + 16,), pad, dtype=dtype, device="cuda")
    t = buf[start:start + M * ld].view(M, ld)[:, :D]
    t.copy_(torch.randn(M, D, generator=g).to(dtype))
    return t


def outside_is_nan(t):
    return int(t._base.isnan().sum()) == t._base.numel() - t.numel()


def case(T, E, k, drop, seed):
    """ids with a share `drop` of pairs without an expert, and what the sort makes of them."""
    g = torch.Generator().manual_seed(seed)
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).int() if T else torch.zeros(0, k).int()
    ids[torch.rand(T, k, generator=g) < drop] = -1
    counts, pos = sort(ids, E)
    return ids.cuda(), counts, pos.cuda(), g


def check_all(b, T, E, k, D, dtype, drop=0.2, p=0.0, ld=None, start=(0, 0, 0, 0), spare=3, add32=False, seed=1):
    """Dispatch and combine, both directions; `spare` rows that no pair has stay as they are."""
    ids, counts, pos, g = case(T, E, k, drop, seed)
    c, q = b.swiglu_moe_sort(ids, E)
    assert torch.equal(c.cpu(), counts) and torch.equal(q, pos)
    N = int(counts.sum())
    x = rows_at(T, D, dtype, g, ld, start[0])
    out = rows_at(N + spare, D, dtype, g, ld, start[1])
    before = out.clone()
    rows = b.swiglu_moe_dispatch_fwd(x, pos, rows=out)
    assert rows is out
    want = before.clone()
    t, j = torch.nonzero(pos >= 0, as_tuple=True)
    want[pos[t, j].long()] = x[t]
    assert torch.equal(rows, want), "dispatch"

    res = rows_at(T, D, F32 if add32 else dtype, g, ld, start[2])
    r64, _ = picked(rows, pos)
    dx = b.swiglu_moe_dispatch_bwd(rows, pos, add=res)
    within(dx, r64.sum(1) + res.double(), (k + 4) * U * (r64.abs().sum(1) + res.double().abs()), "dispatch's gradient")
    dx = b.swiglu_moe_dispatch_bwd(rows, pos)
    within(dx, r64.sum(1), (k + 4) * U * r64.abs().sum(1), "dispatch's gradient alone")

    gates = torch.rand(T, k, generator=g).cuda()
    gates[pos < 0] = float("nan")                          # not read
    step = torch.tensor(-7, dtype=torch.int64, device="cuda")
    kw = dict(p=p, seed=SEED, offset=5, step=step)
    res = rows_at(T, D, dtype, g, ld, start[2])
    w = torch.where(pos >= 0, gates, 0.0).double()[:, :, None]
    terms = r64 * w
    for r in (res, None):
        y = b.swiglu_moe_combine_fwd(rows, pos, gates, residual=r, **kw)
        ref = dropped(terms.sum(1), p, SEED, 5 - 7)
        scale = (k + 4) * U * dropped(terms.abs().sum(1), p, SEED, 5 - 7)
        if r is not None:
            ref, scale = ref + r.double(), scale + (k + 4) * U * r.double().abs()
        within(y, ref, scale, "combine")

    dy = rows_at(T, D, dtype, g, ld, start[3])
    into = rows_at(N + spare, D, dtype, g, ld, start[1])
    before = into.clone()
    drows, dgates = b.swiglu_moe_combine_bwd(dy, rows, pos, gates, drows=into, **kw)
    e = dropped(dy.double(), p, SEED, 5 - 7)
    ref = torch.zeros(T, k, dtype=torch.float64, device="cuda")
    mag = ref.clone()
    ref[t, j], mag[t, j] = (e[t] * r64[t, j]).sum(1), (e[t] * r64[t, j]).abs().sum(1)
    within(dgates, ref, (D / 64 + 40) * U * mag, "dgates")
    want = before.double()
    want[pos[t, j].long()] = e[t] * w[t, j]
    within(drows, want, 3 * U * want.abs(), "drows")
    assert torch.equal(drows[N:], before[N:]), "rows that no pair has"
    assert outside_is_nan(out) and outside_is_nan(into), "elements between the rows"


# tokens, experts, choices, width: one token; one column; fewer than a pack; ragged and odd widths; one pack
# more than a CTA's threads; choices past a register block; wide rows
SHAPES = [(1, 4, 1, 1), (1, 8, 8, 2048), (3, 5, 2, 7), (16, 8, 2, 4096), (37, 6, 3, 8), (33, 40, 7, 1021), (5, 3, 3, 2056),
          (130, 64, 6, 264), (2, 700, 20, 100), (7, 9, 5, 8193), (3, 2, 1, 65536 + 24), (1000, 16, 4, 36),
          (2, 5, 3, 40001), (3, 4, 2, 32771), (70, 16, 9, 130), (2, 1024, 1024, 40), (2, 1024, 1000, 33)]


@pytest.mark.parametrize("dtype", [BF, HF, F32], ids=str)
@pytest.mark.parametrize("T,E,k,D", SHAPES)
def test_there_and_back(b, T, E, k, D, dtype):
    check_all(b, T, E, k, D, dtype)
    check_all(b, T, E, k, D, dtype, drop=0.0, p=0.25, spare=0, add32=True)


@pytest.mark.parametrize("dtype", [BF, F32], ids=str)
@pytest.mark.parametrize("D,ld,start", [(64, 72, (0, 0, 0, 0)), (64, 65, (0, 0, 0, 0)), (61, 64, (0, 0, 0, 0)), (64, 64, (1, 2, 3, 5)),
                                        (1021, 1021, (3, 0, 1, 6)), (515, 600, (7, 7, 7, 7)), (9, 9, (1, 1, 1, 1)),
                                        (64, 64, (0, 1, 0, 0)), (4, 5, (2, 1, 3, 0)), (32768, 32776, (1, 3, 3, 5))])
def test_rows_at_any_place(b, D, ld, start, dtype):
    check_all(b, 19, 6, 3, D, dtype, p=0.5, ld=ld, start=start)
    check_all(b, 19, 6, 3, D, dtype, ld=ld, start=start, add32=True)


@pytest.mark.parametrize("drop,T", [(1.0, 9), (0.0, 0), (1.0, 1)])
def test_no_pairs_and_no_tokens(b, drop, T):
    for dtype in (BF, F32):
        for spare in (0, 2):
            check_all(b, T, 4, 2, 40, dtype, drop=drop, p=0.1, spare=spare)


def test_positions_outside_the_rows_are_no_pairs(b):
    """Whatever pos holds, only rows 0 .. n - 1 are touched."""
    x = torch.randn(3, 24, device="cuda")
    pos = torch.tensor([[0, 4], [-5, 2 ** 31 - 1], [-2 ** 31, 3]], dtype=torch.int32, device="cuda")
    rows = torch.zeros(4, 24, device="cuda")
    b.swiglu_moe_dispatch_fwd(x, pos, rows=rows)
    assert torch.equal(rows[0], x[0]) and torch.equal(rows[3], x[2]) and not rows[1:3].any()
    gates = torch.full((3, 2), float("inf"), device="cuda")
    gates[0, 0] = gates[2, 1] = 1.0
    y = b.swiglu_moe_combine_fwd(rows, pos, gates)
    assert torch.equal(y[0], x[0]) and not y[1].any() and torch.equal(y[2], x[2])
    drows, dgates = b.swiglu_moe_combine_bwd(x, rows, pos, gates, drows=torch.zeros_like(rows))
    assert torch.equal(drows, rows)
    assert not dgates[0, 1].any() and not dgates[1].any() and not dgates[2, 0].any()
    assert torch.equal(b.swiglu_moe_dispatch_bwd(rows, pos), y)


def test_rows_past_32_bit_offsets(b):
    """Rows whose elements lie 2^31 and more past the first, and tokens of more than 2^31 columns in all."""
    D, n = 4096, (1 << 20) + 9
    rows = torch.empty(n, D, dtype=BF, device="cuda")
    x = torch.randn(2, D, device="cuda").to(BF)
    pos = torch.tensor([[n - 1, 0], [1 << 19, n - 2]], dtype=torch.int32, device="cuda")
    b.swiglu_moe_dispatch_fwd(x, pos, rows=rows)
    for t in range(2):
        for r in pos[t].tolist():
            assert torch.equal(rows[r], x[t])
    gates = torch.full((2, 2), 0.5, device="cuda")
    assert torch.equal(b.swiglu_moe_combine_fwd(rows, pos, gates), x)
    dx = b.swiglu_moe_dispatch_bwd(rows, pos)
    assert torch.equal(dx, x + x)
    _, dgates = b.swiglu_moe_combine_bwd(x, rows, pos, gates, drows=rows.new_empty(rows.shape))
    ref = (x.double() ** 2).sum(1, keepdim=True).expand(2, 2)
    within(dgates, ref, (D / 64 + 40) * U * ref, "dgates")
    many = rows.view(-1, 4096)                             # n tokens of one row each, in place
    one = torch.arange(n, dtype=torch.int32, device="cuda")[:, None].contiguous()
    rows.fill_(1.0)
    b.swiglu_moe_combine_fwd(many, one, torch.ones(n, 1, device="cuda"), residual=many, y=(y := torch.empty_like(many)))
    assert bool((y == 2).all())


def test_more_threads_than_a_launch_numbers(b):
    """Past 2^31 packs of 16 bytes (or (pair, pack)s at odd widths) a call is several launches."""
    M, D, seed = (1 << 22) + 5, 4096, 77
    x = torch.ones(M, D, dtype=BF, device="cuda")          # 34 GB, in place
    b.swiglu_mlp_dropout(x, 0.5, seed, y=x)
    for row in (0, (1 << 22) - 3):
        mask, f = keep_mask(8, D, 0.5, seed, 0, row)
        assert torch.equal(x[row:row + 8], (mask * f).to(BF))
    mask, _ = keep_mask(8, D, 0.5, seed, 0, M - 8)
    assert torch.equal(x[M - 8:] != 0, mask)
    del x
    T, k, D = 1 << 16, 1024, 263
    x = torch.randn(T, D, device="cuda").to(BF)
    pos = torch.full((T, k), -1, dtype=torch.int32, device="cuda")
    pos[:, 1000] = torch.arange(T, device="cuda").flip(0)
    assert torch.equal(b.swiglu_moe_dispatch_fwd(x, pos, T), x.flip(0))


def test_in_place(b):
    for dtype, D in ((BF, 64), (HF, 61), (F32, 61)):
        ids, counts, pos, g = case(21, 5, 2, 0.3, 4)
        rows = rows_at(int(counts.sum()), D, dtype, g)
        gates = torch.rand(21, 2, generator=g).cuda()
        res = rows_at(21, D, dtype, g)
        want = b.swiglu_moe_combine_fwd(rows, pos, gates, residual=res, p=0.3, seed=1)
        want_dx = b.swiglu_moe_dispatch_bwd(rows, pos, add=res)
        y = res.clone()
        assert b.swiglu_moe_combine_fwd(rows, pos, gates, residual=y, p=0.3, seed=1, y=y) is y and torch.equal(y, want)
        y = res.clone()
        assert torch.equal(b.swiglu_moe_dispatch_bwd(rows, pos, add=y, dx=y), want_dx)


def test_the_same_bits_on_every_run_and_on_another_stream(b):
    ids, counts, pos, g = case(700, 16, 5, 0.1, 5)
    rows, dy = rows_at(int(counts.sum()), 515, BF, g), rows_at(700, 515, BF, g)
    gates = torch.rand(700, 5, generator=g).cuda()

    def calls():
        return (*b.swiglu_moe_sort(ids, 16), b.swiglu_moe_combine_fwd(rows, pos, gates, p=0.1, seed=3),
                *b.swiglu_moe_combine_bwd(dy, rows, pos, gates, p=0.1, seed=3), b.swiglu_moe_dispatch_bwd(rows, pos))

    want = calls()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = calls()
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    assert all(torch.equal(p, q) for p, q in zip(calls(), want))


# ------------------------------------------------------------------------------ sort

@pytest.mark.parametrize("n,E", [(0, 3), (1, 1), (31, 4), (1025, 1024), (4096, 64), (8193, 7), (100003, 129), (1 << 20, 682)])
def test_sort(b, n, E):
    g = torch.Generator().manual_seed(n)
    ids = torch.randint(-2, E + 2, (n,), generator=g).int()
    if n > 4000:                                           # runs of one expert, an empty one
        ids[1000:3000] = E // 2
        ids[ids == E - 1] = 0
    counts, pos = b.swiglu_moe_sort(ids.cuda(), E)
    want_c, want_p = sort(torch.where((ids >= 0) & (ids < E), ids, -1), E)
    assert torch.equal(counts.cpu(), want_c) and torch.equal(pos.cpu(), want_p)


@pytest.mark.parametrize("value", [0, 5, -1])
def test_sort_of_one_value(b, value):
    counts, pos = b.swiglu_moe_sort(torch.full((3333, 4), value, dtype=torch.int32, device="cuda"), 6)
    n = 3333 * 4
    assert counts.tolist() == [n if e == value else 0 for e in range(6)]
    want = torch.arange(n, dtype=torch.int32, device="cuda").view(3333, 4)
    assert torch.equal(pos, want if value >= 0 else torch.full_like(want, -1))


# ------------------------------------------------------------------------------ dropout

@pytest.mark.parametrize("dtype", [BF, HF, F32], ids=str)
@pytest.mark.parametrize("M,D,ld,start", [(1, 1, 1, 0), (1, 9, 9, 0), (5, 64, 64, 0), (5, 64, 64, 3), (128, 256, 256, 0),
                                          (37, 1021, 1021, 0), (3, 20001, 20010, 1), (700, 24, 25, 5)])
def test_dropout(b, M, D, ld, start, dtype):
    g = torch.Generator().manual_seed(D)
    x, r = rows_at(M, D, dtype, g, ld, start), rows_at(M, D, dtype, g)
    for p, seed, offset, step in [(0.5, 0, 0, None), (0.1, SEED, 2 ** 64 - 1, 2), (0.999, 1, 2 ** 40, -3), (1.0, 5, 5, None), (0.0, 1, 1, 1),
                                  (1 / 3, 2 ** 63, 1, 2 ** 62)]:
        t = None if step is None else torch.tensor(step, dtype=torch.int64, device="cuda")
        at = offset + (step or 0)
        for res in (None, r):
            y = b.swiglu_mlp_dropout(x, p, seed, offset, t, residual=res)
            kept = dropped(x.double(), p, seed, at)
            ref = kept if res is None else kept + res.double()
            within(y, ref, 3 * U * (kept.abs() + ref.abs()), f"p {p}")
            if p == 1.0:
                assert torch.equal(y, torch.zeros_like(y) if res is None else res)
        for place in (x, r):
            buf = place.clone(memory_format=torch.preserve_format)
            want = b.swiglu_mlp_dropout(x, p, seed, offset, t, residual=r)
            got = b.swiglu_mlp_dropout(buf if place is x else x, p, seed, offset, t, residual=buf if place is r else r, y=buf)
            assert got is buf and torch.equal(got, want)


def test_dropped_elements_do_not_count_whatever_they_hold(b):
    x = torch.full((64, 96), float("nan"), device="cuda", dtype=BF)
    y = b.swiglu_mlp_dropout(x, 0.5, 11)
    share = y.isnan().float().mean().item()
    assert bool((y.isnan() | (y == 0)).all()) and abs(share - 0.5) < 5 * 0.5 / (64 * 96) ** 0.5
    assert torch.equal(b.swiglu_mlp_dropout(x, 1.0, 11), torch.zeros_like(x))


def test_masks_differ_by_seed_offset_and_row(b):
    x = torch.ones(64, 512, device="cuda")
    masks = [b.swiglu_mlp_dropout(x, 0.25, s, o) != 0 for s, o in [(0, 0), (1, 0), (0, 1), (1 << 32, 0), (0, 1 << 32)]]
    n = x.numel()
    for i, m in enumerate(masks):
        assert abs(m.float().mean().item() - 0.75) < 5 * (0.75 * 0.25 / n) ** 0.5
        for other in masks[:i]:                            # independent: equal with chance 0.625
            assert abs((m == other).float().mean().item() - 0.625) < 5 * (0.625 * 0.375 / n) ** 0.5
    a, c = masks[0][:-1], masks[0][1:]
    assert abs((a == c).float().mean().item() - 0.625) < 5 * (0.625 * 0.375 / a.numel()) ** 0.5


def test_a_graph_with_a_step_has_another_mask_on_every_replay(b):
    x, r = torch.ones(33, 200, device="cuda", dtype=BF), torch.zeros(33, 200, device="cuda", dtype=BF)
    ids, counts, pos, g = case(33, 4, 2, 0.0, 6)
    rows, gates = rows_at(66, 200, BF, g), torch.rand(33, 2, generator=g).cuda()
    step = torch.zeros((), dtype=torch.int64, device="cuda")

    def calls(step, offset):
        return (*b.swiglu_moe_gate_fwd(gates, 1), *b.swiglu_moe_sort(ids, 4), b.swiglu_moe_dispatch_fwd(x, pos),
                b.swiglu_moe_combine_fwd(rows, pos, gates, residual=r, p=0.5, seed=9, offset=offset, step=step),
                *b.swiglu_moe_combine_bwd(x, rows, pos, gates, p=0.5, seed=9, offset=offset, step=step),
                b.swiglu_mlp_dropout(x, 0.5, 9, offset, step), b.swiglu_moe_gate_bwd(gates, pos[:, :1].contiguous(), gates[:, :1].contiguous(), gates[:, 1:].contiguous()))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls(step, 3)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step += 1
        out = calls(step, 3)
    step.zero_()
    for i in (1, 2, 3):
        graph.replay()
        want = calls(None, 3 + i)
        assert step.item() == i and all(torch.equal(p, q) for p, q in zip(out, want))

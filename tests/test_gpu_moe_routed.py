"""GPU tests of the routed MoE layer for a few tokens (swiglu_moe_routed_fwd) against fp64 torch.

Tolerances.  y: the framework's parity bar (helpers.parity); h and y are each rounded to
bf16 once, about 1.7e-3 of the norm apiece.  Gates: a lane adds D / 32 products of a logit in
sequence and 5 shuffle steps follow, so a logit is off by at most (D / 32 + 6) u of the sum of
its products' magnitudes (u = 2^-24), and a gate by twice the largest such error plus 64 u for
the exponentials and their sums.  Chosen ids must be the fp64 ones wherever the fp64 logits
around the choice are further apart than that.
"""
import pytest
import torch

from helpers import ensure_library, parity

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
bf = torch.bfloat16


@pytest.fixture(scope="module")
def b():
    ensure_library()
    from bwd_gemm_epilogue_gb300 import binding
    binding.lib()
    return binding


def draw(T, E, D, H, Dout, seed, router=bf):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s, std=1.0: (std * torch.randn(s, generator=g))  # noqa: E731
    return dict(x=n(T, D).to(bf).cuda(), Wr=n(E, D, std=D ** -0.5).to(router).cuda(),
                W1=n(E, 2 * H, D, std=D ** -0.5).to(bf).cuda(), W2=n(E, Dout, H, std=H ** -0.5).to(bf).cuda(),
                r=n(T, Dout).to(bf).cuda())


def experts_ref(t, ids, gates, residual):
    """y in fp64 for given choices."""
    H = t["W2"].shape[2]
    x = t["x"].double()
    y = residual.double() if residual is not None else torch.zeros(x.shape[0], t["W2"].shape[1], device="cuda",
                                                                   dtype=torch.float64)
    for e in sorted(set(ids.flatten().tolist())):
        at, j = torch.nonzero(ids == e, as_tuple=True)
        z = x[at] @ t["W1"][e].double().T
        h = z[:, :H] * z[:, H:] * torch.sigmoid(z[:, H:])
        y = y.index_add(0, at, (h @ t["W2"][e].double().T) * gates[at, j].double()[:, None])
    return y


def check(b, t, k, renorm, residual, **kw):
    y, ids, gates = b.swiglu_moe_routed_fwd(t["x"], t["Wr"], t["W1"], t["W2"], k, renormalize=renorm,
                                            residual=residual, **kw)
    x, w = t["x"].double(), t["Wr"].double()
    logits = x @ w.T
    err = (x.shape[1] / 32 + 6) * U * (x.abs() @ w.abs().T).max(1, keepdim=True).values
    order = torch.argsort(logits, dim=1, descending=True, stable=True)
    ranked = torch.gather(logits, 1, order)
    gap = torch.full_like(ranked, float("inf"))
    gap[:, 1:] = ranked[:, :-1] - ranked[:, 1:]
    close = gap <= 2 * err
    clear = ~(close | torch.nn.functional.pad(close[:, 1:], (0, 1)))[:, :k]
    assert bool((ids == order[:, :k])[clear].all())
    assert clear.float().mean() > 0.9
    for row in ids.tolist():
        assert len(set(row)) == k and all(0 <= e < logits.shape[1] for e in row)
    own = torch.gather(logits, 1, ids.long())
    want = torch.exp(own - torch.logsumexp(own if renorm else logits, 1, keepdim=True))
    assert bool(((gates.double() - want).abs() <= (2 * err + 64 * U) * want + 1e-37).all())
    parity(y, experts_ref(t, ids, gates, residual).cpu().numpy(), "y")
    return y, ids, gates


# (T, E, D, H, Dout, k): one token; every token on every expert; one expert; widths of one
# group of 8; k steps that end inside 64 and inside 32; 8-, 16-, 32- and 64-token tiles;
# more experts than a warp, than chosen; the largest T, E and k
CASES = [(1, 8, 256, 512, 256, 2), (1, 64, 264, 136, 248, 8), (3, 1, 64, 8, 8, 1), (2, 2, 8, 8, 16, 2),
         (5, 4, 72, 40, 24, 4), (9, 3, 200, 104, 136, 2), (17, 2, 128, 64, 64, 1), (33, 2, 96, 72, 40, 2),
         (64, 1, 136, 200, 72, 1), (64, 5, 520, 264, 264, 5), (31, 33, 256, 64, 128, 3), (64, 128, 128, 64, 128, 16),
         (7, 682, 64, 16, 32, 4), (40, 16, 1032, 328, 1000, 2), (16, 8, 512, 1024, 5000, 2)]


@pytest.mark.parametrize("T,E,D,H,Dout,k", CASES)
@pytest.mark.parametrize("renorm,add", [(True, False), (False, True)])
def test_matches_fp64(b, T, E, D, H, Dout, k, renorm, add):
    t = draw(T, E, D, H, Dout, seed=T + E + D)
    check(b, t, k, renorm, t["r"] if add else None)


def test_fp32_router(b):
    t = draw(12, 20, 264, 64, 64, 3, router=torch.float32)
    check(b, t, 4, True, None)


def test_ties_go_to_the_lowest_index(b):
    t = draw(10, 40, 128, 32, 64, 5)
    t["Wr"][:] = t["Wr"][7]                                  # every expert ties
    _, ids, gates = b.swiglu_moe_routed_fwd(t["x"], t["Wr"], t["W1"], t["W2"], 5)
    assert torch.equal(ids.cpu(), torch.arange(5, dtype=torch.int32).expand(10, 5))
    assert torch.allclose(gates, torch.full_like(gates, 0.2), rtol=1e-6)
    t = draw(10, 40, 128, 32, 64, 6)
    t["Wr"][31] = t["Wr"][3]                                 # one pair, across the lanes of a warp
    t["Wr"][35] = t["Wr"][3]
    _, ids, _ = b.swiglu_moe_routed_fwd(t["x"], t["Wr"], t["W1"], t["W2"], 16)
    for row in ids.tolist():
        if 31 in row:
            assert row.index(3) == row.index(31) - 1
        if 35 in row:
            assert row.index(31) == row.index(35) - 1


def test_lopsided_gates_and_saturated_activations(b):
    """Logits in the hundreds (all weight on one expert) and gates far into both tails of silu."""
    t = draw(6, 9, 256, 128, 64, 8)
    t["Wr"] *= 200
    t["W1"][:, 128:] *= 60
    check(b, t, 3, True, None)


def test_non_finite_tokens_stay_their_own(b):
    t = draw(20, 6, 200, 64, 104, 9)
    clean = b.swiglu_moe_routed_fwd(t["x"], t["Wr"], t["W1"], t["W2"], 2)
    x = t["x"].clone()
    x[3, 5], x[11, 199], x[12] = float("nan"), float("inf"), float("-inf")
    y, ids, gates = b.swiglu_moe_routed_fwd(x, t["Wr"], t["W1"], t["W2"], 2)
    assert b.swiglu_mlp_device_status() == 0
    bad = torch.tensor([i in (3, 11, 12) for i in range(20)], device="cuda")
    assert bool(y[bad].isnan().all()) and bool(gates[bad].isnan().all())
    assert bool(((ids >= 0) & (ids < 6)).all())
    for got, want in zip((y, ids, gates), clean):
        assert torch.equal(got[~bad], want[~bad])


def test_unchosen_experts_are_not_read_into_the_result(b):
    """Weights of NaN in every expert that no token chose change nothing."""
    t = draw(2, 50, 128, 64, 64, 10)
    y, ids, _ = b.swiglu_moe_routed_fwd(t["x"], t["Wr"], t["W1"], t["W2"], 3)
    rest = torch.ones(50, dtype=torch.bool, device="cuda")
    rest[ids.long().flatten()] = False
    t["W1"][rest], t["W2"][rest] = float("nan"), float("nan")
    assert torch.equal(b.swiglu_moe_routed_fwd(t["x"], t["Wr"], t["W1"], t["W2"], 3)[0], y)


def test_no_tokens(b):
    t = draw(1, 4, 64, 64, 64, 1)
    y, ids, gates = b.swiglu_moe_routed_fwd(t["x"][:0], t["Wr"], t["W1"], t["W2"], 2)
    assert y.shape == (0, 64) and ids.shape == (0, 2) and gates.shape == (0, 2)


def test_agrees_with_the_grouped_layer(b):
    """The grouped layer (swiglu_moe_fwd) on the same choices, gathered and combined in torch."""
    T, k = 24, 3
    t = draw(T, 10, 264, 136, 264, 11)
    y, ids, gates = b.swiglu_moe_routed_fwd(t["x"], t["Wr"], t["W1"], t["W2"], k)
    order = torch.argsort(ids.flatten(), stable=True)
    counts = torch.bincount(ids.flatten(), minlength=10).tolist()
    _, rows = b.swiglu_moe_fwd(t["x"].repeat_interleave(k, 0)[order].contiguous(), t["W1"], t["W2"], counts)
    back = torch.empty_like(rows)
    back[order] = rows
    ref = (back.double().reshape(T, k, -1) * gates.double()[..., None]).sum(1)
    parity(y, ref.cpu().numpy(), "y", rel_fro=1e-2, max_abs_frac=4e-2)     # two roundings on either side


def test_same_bits_every_run_on_another_stream_and_in_a_graph(b):
    t = draw(30, 12, 512, 264, 520, 12)
    args = (t["x"], t["Wr"], t["W1"], t["W2"], 4)
    want = b.swiglu_moe_routed_fwd(*args, residual=t["r"])
    for got, ref in zip(b.swiglu_moe_routed_fwd(*args, residual=t["r"]), want):
        assert torch.equal(got, ref)
    y, ids, gates = (torch.empty_like(v) for v in want)
    ws = torch.empty(b.swiglu_moe_routed_fwd_workspace_size(30, 264, 520, 4), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            b.swiglu_moe_routed_fwd(*args, residual=t["r"], y=y, ids=ids, gates=gates, workspace=ws)
        for _ in range(2):
            y.zero_(), ids.fill_(-1), gates.zero_()
            graph.replay()
    torch.cuda.current_stream().wait_stream(side)
    for got, ref in zip((y, ids, gates), want):
        assert torch.equal(got, ref)


def test_weights_past_32_bit_offsets(b):
    """An expert whose weights start beyond 2^31 elements."""
    E, D, H = 40, 4096, 8192
    W1 = torch.empty(E, 2 * H, D, dtype=bf, device="cuda")
    W2 = torch.empty(E, D, H, dtype=bf, device="cuda")
    t = draw(2, E, D, 8, 8, 13)
    g = torch.Generator(device="cuda").manual_seed(2)
    for e in (1, 39):
        W1[e].normal_(0, D ** -0.5, generator=g)
        W2[e].normal_(0, H ** -0.5, generator=g)
    t["W1"], t["W2"] = W1, W2
    t["Wr"].zero_()
    t["Wr"][1, :8], t["Wr"][39, :8] = 1.0, 1.0
    t["x"][:, :8] = 1.0
    y, ids, gates = b.swiglu_moe_routed_fwd(t["x"], t["Wr"], W1, W2, 2)
    assert ids.tolist() == [[1, 39]] * 2
    parity(y, experts_ref(t, ids, gates, None).cpu().numpy(), "y")

"""GPU tests of the C entry points called from two threads at once, for launches of one kernel with different
amounts of shared memory, past what a kernel may have without leave."""
import ctypes
import threading

import pytest
import torch

from test_gpu_tokens import BF, b  # noqa: F401

pytestmark = pytest.mark.gpu
TURNS = 10000


def c(v):
    """A tensor or a whole number as ctypes has it, made once: the threads shall spend their time in the calls."""
    return ctypes.c_void_p(v.data_ptr()) if isinstance(v, torch.Tensor) else ctypes.c_int64(v) if isinstance(v, int) else v


def at_once(entry, calls):
    """calls: (arguments, outputs).  Each is made once alone, then all TURNS times, a thread and a stream each."""
    want = []
    for args, outs in calls:
        assert entry(*map(c, args), None) == 0
        torch.cuda.synchronize()
        want.append([t.clone() for t in outs])
        for t in outs:
            t.zero_()
    torch.cuda.synchronize()
    statuses, go = [{} for _ in calls], threading.Barrier(len(calls))

    def run(i, args):
        stream = torch.cuda.Stream()
        args = [*map(c, args), ctypes.c_void_p(stream.cuda_stream)]
        go.wait()
        for turn in range(TURNS):
            st = entry(*args)
            statuses[i][st] = statuses[i].get(st, 0) + 1
            if turn % 64 == 63:                            # few launches queued: what is looked for is at the call
                stream.synchronize()
        stream.synchronize()

    threads = [threading.Thread(target=run, args=(i, args)) for i, (args, _) in enumerate(calls)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert statuses == [{0: TURNS}] * len(calls)
    for (_, outs), alone in zip(calls, want):
        assert all(torch.equal(p, q) for p, q in zip(outs, alone))


def test_sorts(b):  # noqa: F811
    g = torch.Generator().manual_seed(1)
    calls = []
    for n, E in ((256, 1024), (1024, 1024)):               # 74 and 205 KB
        ids = torch.randint(0, E, (n,), generator=g).int().cuda()
        counts, pos = torch.empty(E, dtype=torch.int32, device="cuda"), torch.empty_like(ids)
        calls.append(((ids, counts, pos, n, E), (counts, pos)))
    at_once(b.lib().swiglu_moe_sort, calls)


def test_layer_norms_forward(b):  # noqa: F811
    calls = []
    for D in (7001, 12001):                                # odd rows, whose parameters go through 56 and 96 KB
        x, y = torch.randn(3, D, device="cuda").to(BF), torch.empty(3, D, dtype=BF, device="cuda")
        w, stats = torch.randn(2, D, device="cuda").to(BF), torch.empty(2, 3, device="cuda")
        calls.append(((x, D, None, 0, w[0], w[1], y, D, None, 0, stats[0], stats[1], 3, D, ctypes.c_float(1e-5), ctypes.c_int(0),
                       ctypes.c_int(0)), (y, stats)))
    at_once(b.lib().swiglu_mlp_layer_norm_fwd, calls)


def test_layer_norms_backward(b):  # noqa: F811
    calls = []
    M = 480
    for D in (2048, 3584):                                 # 74 and 111 KB: rows in flight, and gamma
        dy, s, dx = (torch.randn(M, D, device="cuda").to(BF) for _ in range(3))
        w, stats = torch.randn(3, D, device="cuda").to(BF), torch.rand(2, M, device="cuda")
        need = b.swiglu_mlp_layer_norm_bwd_workspace_size(M, D)
        calls.append(((dy, D, s, D, w[0], stats[0], stats[1], None, 0, dx, D, w[1], w[2], M, D, ctypes.c_int(0), ctypes.c_int(0),
                       torch.empty(need, dtype=torch.uint8, device="cuda"), ctypes.c_size_t(need)), (dx, w[1:])))
    at_once(b.lib().swiglu_mlp_layer_norm_bwd, calls)


@pytest.mark.parametrize("tokens", [(1, 32), (2, 9), (33, 64)])
def test_routed_layers(b, tokens):  # noqa: F811
    """The down products' sums take 1 KB of shared memory for each token."""
    g = torch.Generator().manual_seed(2)
    E, D, H, k = 4, 64, 64, 1
    weights = [(torch.randn(s, generator=g) * s[-1] ** -0.5).to(BF).cuda() for s in ((E, D), (E, 2 * H, D), (E, D, H))]
    calls = []
    for T in tokens * 2:
        x, y = torch.randn(T, D, generator=g).to(BF).cuda(), torch.empty(T, D, dtype=BF, device="cuda")
        ids, gates = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
        need = b.swiglu_moe_routed_fwd_workspace_size(T, H, D, k)
        calls.append(((x, *weights, None, y, ids, gates, T, E, D, H, D, k, ctypes.c_int(1), ctypes.c_int(0),
                       torch.empty(need, dtype=torch.uint8, device="cuda"), ctypes.c_size_t(need)), (y, ids, gates)))
    at_once(b.lib().swiglu_moe_routed_fwd, calls)

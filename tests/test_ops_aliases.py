"""Refusals of overlapping outputs by the operators' C entry points (CPU only: the checks come before
anything reaches a device)."""
import ctypes

from test_ops_checks import A, INVALID, b  # noqa: F401


def test_one_place_for_both_outputs_of_the_norm_is_refused(b):  # noqa: F811
    L = b.lib()
    assert L.swiglu_mlp_layer_norm_fwd(A, 64, 2 * A, 64, A, A, 3 * A, 64, 3 * A, 64, A, A, 4, 64, 1e-5, 0, 2, None) == INVALID
    assert b"the same" in L.swiglu_mlp_last_error_detail()


def clip(L, ins, outs, counts, types):
    n = len(ins)
    i64, ptr = ctypes.c_int64 * n, ctypes.c_void_p * n
    return L.swiglu_mlp_clip_grads(ptr(*ins), ptr(*outs), i64(*counts), (ctypes.c_int * n)(*types), n, 1.0, 1e-6, A, A,
                                   1 << 30, None)


def test_overlapping_outputs_of_the_clipping_are_refused(b):  # noqa: F811
    """One gradient twice, parts of one another, an output in another gradient's place; lists of the
    small and of the large table."""
    L = b.lib()
    for spare in (0, 100):
        more = [A + 0x1000 * (10 + i) for i in range(spare)]
        rest = [100] * spare, [0] * spare
        for ins, outs, counts, types in [
            ((A, A), (A, A), (5, 5), (2, 2)),                                    # in place, listed twice
            ((A, A + 16), (A, A + 16), (5, 5), (2, 2)),                          # 20 bytes from A: 4 shared
            ((A, 2 * A), (3 * A, 3 * A + 8), (5, 5), (0, 0)),                    # outputs apart from the inputs
            ((A, 2 * A), (2 * A, A), (5, 5), (0, 0)),                            # in each other's place
            ((A,), (A + 2,), (5,), (0,)),                                        # shifted against its own input
            ((A, 2 * A, 3 * A), (4 * A, 5 * A, A + 4), (3, 4, 5), (0, 0, 0)),
        ]:
            assert clip(L, (*ins, *more), (*outs, *more), (*counts, *rest[0]), (*types, *rest[1])) == INVALID, (ins, outs)
            assert b"overlap" in L.swiglu_mlp_last_error_detail()
            assert clip(L, (*more, *ins), (*more, *outs), (*rest[0], *counts), (*rest[1], *types)) == INVALID, (ins, outs)


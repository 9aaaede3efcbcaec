"""Refusals of overlapping outputs by the operators' C entry points (CPU only: the checks come before
anything reaches a device)."""
from test_ops_checks import A, INVALID, b  # noqa: F401


def test_one_place_for_both_outputs_of_the_norm_is_refused(b):  # noqa: F811
    L = b.lib()
    assert L.swiglu_mlp_layer_norm_fwd(A, 64, 2 * A, 64, A, A, 3 * A, 64, 3 * A, 64, A, A, 4, 64, 1e-5, 0, 2, None) == INVALID
    assert b"the same" in L.swiglu_mlp_last_error_detail()

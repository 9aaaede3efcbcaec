"""Refusals, by the layer norm's C entry points, of outputs in an input's place with another row stride, whose
rows would be written over others that have yet to be read (CPU only: the checks come before anything reaches
a device)."""
from test_ops_checks import A, b  # noqa: F401
from test_tokens_aliases import refused  # noqa: F401


def fwd(x, ldx, r, ldr, y, ldy, s, lds, M=4):
    return "swiglu_mlp_layer_norm_fwd", x, ldx, r, ldr, None, None, y, ldy, s, lds, 8 * A, 9 * A, M, 64, 1e-5, 0, 2


def bwd(dy, lddy, s, lds, skip, ldskip, dx, lddx, M=4):
    return ("swiglu_mlp_layer_norm_bwd", dy, lddy, s, lds, None, 8 * A, 9 * A, skip, ldskip, dx, lddx, None, None, M, 64, 0, 2,
            16 * A, 1 << 30)


def test_rows_of_another_stride(refused):  # noqa: F811
    for place in ((A, 64, 2 * A, 64, A, 72, 3 * A, 64), (A, 64, 2 * A, 64, 3 * A, 64, A, 72), (A, 64, 2 * A, 72, 2 * A, 64, 3 * A, 64),
                  (A, 64, 2 * A, 64, 3 * A, 64, 2 * A, 72), (A, 72, None, 0, A, 64, None, 0)):
        assert refused(*fwd(*place)), place
        assert not refused(*fwd(*place, M=1)), place
    for place in ((A, 64, 2 * A, 64, None, 0, A, 72), (A, 64, 2 * A, 64, 3 * A, 64, 2 * A, 72), (A, 64, 2 * A, 64, 3 * A, 72, 3 * A, 64)):
        assert refused(*bwd(*place)), place
        assert not refused(*bwd(*place, M=1)), place


def test_the_same_rows(refused):  # noqa: F811
    assert not refused(*fwd(A, 72, 2 * A, 80, A, 72, 2 * A, 80)) and not refused(*fwd(A, 72, 2 * A, 80, 2 * A, 80, A, 72))
    assert not refused(*fwd(A, 72, None, 0, 2 * A, 64, None, 0))
    assert not refused(*bwd(A, 72, 2 * A, 64, 3 * A, 80, A, 72)) and not refused(*bwd(A, 72, 2 * A, 64, 3 * A, 80, 3 * A, 80))

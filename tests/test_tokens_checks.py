"""Refusals of the operators of include/swiglu_tokens.h, and the counter-based generator of their tests
against published values (CPU only: the checks come before anything reaches a device)."""
import re

import pytest
import torch

from helpers import ROOT
from test_ops_checks import A, CUDA, INVALID, MISALIGNED, SHAPE, b, z  # noqa: F401
from tokens_reference import philox

i32, f32 = torch.int32, torch.float32
T, E, k, D, N = 6, 9, 3, 40, 11


def test_generator_of_the_tests():
    """Known answers of Philox4x32-10 that its authors publish with it."""
    ones = 0xffffffff
    assert philox([[0, 0, 0, 0]], (0, 0)).tolist() == [[0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8]]
    assert philox([[ones] * 4], (ones, ones)).tolist() == [[0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd]]


def test_header_and_binding_agree(b):  # noqa: F811
    src = re.sub(r"/\*.*?\*/", "", open(f"{ROOT}/include/swiglu_tokens.h").read(), flags=re.S)
    names = set(re.findall(r"\b(swiglu_\w+)\s*\(", src))
    assert len(names) == 8
    for n in names:
        assert hasattr(b.lib(), n) and n in b.SIGNATURES


def test_legal_calls_pass_every_check_but_the_device(b):  # noqa: F811
    l, ids, q, x, rows = z(T, E), z(T, k, dtype=i32), z(T, k, dtype=f32), z(T, D), z(N, D)
    for call in (lambda: b.swiglu_moe_gate_fwd(l, k), lambda: b.swiglu_moe_gate_bwd(l, ids, q, q),
                 lambda: b.swiglu_moe_sort(ids, E), lambda: b.swiglu_moe_dispatch_fwd(x, ids),
                 lambda: b.swiglu_moe_dispatch_fwd(x, ids, N), lambda: b.swiglu_moe_dispatch_bwd(rows, ids, add=x.float()),
                 lambda: b.swiglu_moe_combine_fwd(rows, ids, q, residual=x, p=0.5, step=torch.tensor(3)),
                 lambda: b.swiglu_moe_combine_bwd(x, rows, ids, q), lambda: b.swiglu_mlp_dropout(x, 0.1, 2 ** 64 - 1, residual=x),
                 lambda: b.moe_gate(l.view(2, 3, E), k), lambda: b.dropout(x, 0.5, 1)):
        with pytest.raises(ValueError, match=CUDA):
            call()


def test_wrong_tensors_are_refused_by_name(b):  # noqa: F811
    l, ids, q, x, rows = z(T, E), z(T, k, dtype=i32), z(T, k, dtype=f32), z(T, D), z(N, D)
    for call, err, match in [
        (lambda: b.swiglu_moe_gate_fwd(z(E), k), ValueError, "logits: shape"),
        (lambda: b.swiglu_moe_gate_fwd(l.double(), k), TypeError, "logits: torch.float64"),
        (lambda: b.swiglu_moe_gate_fwd(z(E, T).T, k), ValueError, "logits: each row"),
        (lambda: b.swiglu_moe_gate_fwd(l, 0), ValueError, "top_k: 0"),
        (lambda: b.swiglu_moe_gate_fwd(l, E + 1), ValueError, "top_k: 10"),
        (lambda: b.swiglu_moe_gate_fwd(l, k, ids=ids.long()), TypeError, "ids: torch.int64"),
        (lambda: b.swiglu_moe_gate_bwd(l, ids[:, :2], q, q), ValueError, "ids: must be contiguous"),
        (lambda: b.swiglu_moe_gate_bwd(l, ids, q[1:], q), ValueError, "gates: shape"),
        (lambda: b.swiglu_moe_gate_bwd(l, ids, q, q.bfloat16()), TypeError, "dgates: torch.bfloat16"),
        (lambda: b.swiglu_moe_gate_bwd(l, ids, q, q, dlogits=l.float()), TypeError, "dlogits: torch.float32"),
        (lambda: b.swiglu_moe_sort(ids.long(), E), TypeError, "ids: torch.int64"),
        (lambda: b.swiglu_moe_sort(ids, E, counts=z(E + 1, dtype=i32)), ValueError, "counts: shape"),
        (lambda: b.swiglu_moe_dispatch_fwd(x, ids[1:].contiguous()), ValueError, "pos: shape"),
        (lambda: b.swiglu_moe_dispatch_fwd(x, ids.float()), TypeError, "pos: torch.float32"),
        (lambda: b.swiglu_moe_dispatch_fwd(x, ids, -1), ValueError, "n_rows: -1"),
        (lambda: b.swiglu_moe_dispatch_fwd(x, ids, N + 1, rows=rows), ValueError, "n_rows: 12"),
        (lambda: b.swiglu_moe_dispatch_fwd(x, ids, rows=rows.float()), TypeError, "rows: torch.float32"),
        (lambda: b.swiglu_moe_dispatch_bwd(rows, ids, add=z(T, D + 1)), ValueError, "add: shape"),
        (lambda: b.swiglu_moe_dispatch_bwd(rows, ids, add=x.half()), TypeError, "add: torch.float16"),
        (lambda: b.swiglu_moe_combine_fwd(rows, ids, q, residual=x.float()), TypeError, "residual: torch.float32"),
        (lambda: b.swiglu_moe_combine_fwd(rows, ids, q.T.contiguous().T), ValueError, "gates: must be contiguous"),
        (lambda: b.swiglu_moe_combine_fwd(rows, ids, q, seed=-1), ValueError, "seed: -1"),
        (lambda: b.swiglu_moe_combine_fwd(rows, ids, q, seed=1.5), TypeError, "integer"),
        (lambda: b.swiglu_moe_combine_fwd(rows, ids, q, step=torch.zeros(1, dtype=torch.int64)), ValueError, "step: shape"),
        (lambda: b.swiglu_moe_combine_bwd(z(T, D + 8), rows, ids, q), ValueError, "dy: shape"),
        (lambda: b.swiglu_moe_combine_bwd(x, rows, ids, q, drows=z(N + 1, D)), ValueError, "drows: shape"),
        (lambda: b.swiglu_mlp_dropout(x, 0.5, 1 << 64), ValueError, "seed: "),
        (lambda: b.swiglu_mlp_dropout(x, 0.5, 1, step=torch.tensor(1, dtype=i32)), TypeError, "step: torch.int32"),
        (lambda: b.swiglu_mlp_dropout(x, 0.5, 1, residual=z(T, D - 1)), ValueError, "residual: shape"),
    ]:
        with pytest.raises(err, match=match):
            call()


def test_gate_and_sort_argument_errors(b):  # noqa: F811
    L = b.lib()

    def fwd(l=A, ld=64, ids=A, gates=A, T=4, E=64, k=2, type=0):
        return L.swiglu_moe_gate_fwd(l, ld, ids, gates, T, E, k, 1, type, None)

    assert fwd(T=0) == 0 and fwd(T=0, l=None) == 0
    assert fwd(T=-1) == INVALID and fwd(E=0) == INVALID and fwd(k=0) == INVALID and fwd(k=65) == INVALID
    assert fwd(T=1 << 31) == SHAPE and fwd(E=1025, ld=1025) == SHAPE
    assert fwd(type=3) == INVALID and fwd(l=None) == INVALID and fwd(ids=None) == INVALID and fwd(ld=63) == INVALID
    assert fwd(l=A + 1) == MISALIGNED and fwd(gates=A + 2) == MISALIGNED
    assert b"gate" in L.swiglu_mlp_last_error_detail()

    def bwd(l=A, ld=64, ids=A, q=A, dq=A, d=A, ldd=64, T=4, E=64, k=2, renorm=0, type=0):
        return L.swiglu_moe_gate_bwd(l, ld, ids, q, dq, d, ldd, T, E, k, renorm, type, None)

    assert bwd(T=0) == 0 and bwd(l=None) == INVALID and bwd(dq=None) == INVALID and bwd(d=None, renorm=1) == INVALID
    assert bwd(ld=63) == INVALID and bwd(ldd=63, renorm=1) == INVALID and bwd(d=A + 1) == MISALIGNED

    def sort(ids=A, counts=A, pos=A, n=10, E=4):
        return L.swiglu_moe_sort(ids, counts, pos, n, E, None)

    assert sort(n=-1) == INVALID and sort(E=0) == INVALID and sort(E=1025) == SHAPE and sort(n=1 << 31) == SHAPE
    assert sort(ids=None) == INVALID and sort(counts=None, n=0) == INVALID and sort(pos=A + 2) == MISALIGNED


def test_rows_argument_errors(b):  # noqa: F811
    L = b.lib()

    def there(x=A, ldx=64, pos=A, rows=A, ldr=64, T=4, D=64, k=2, n=8, type=0):
        return L.swiglu_moe_dispatch_fwd(x, ldx, pos, rows, ldr, T, D, k, n, type, None)

    assert there(T=0) == 0 and there(n=0) == 0
    assert there(T=-1) == INVALID and there(D=0) == INVALID and there(k=0) == INVALID and there(n=-1) == INVALID
    assert there(T=1 << 31) == SHAPE and there(n=1 << 31) == SHAPE and there(D=1 << 28, ldx=1 << 28, ldr=1 << 28) == SHAPE
    assert there(k=1025) == SHAPE and there(D=1 << 22, ldx=1 << 22, ldr=1 << 22, k=512) == SHAPE
    assert there(x=None) == INVALID and there(ldr=63) == INVALID and there(type=7) == INVALID
    assert there(rows=A + 1) == MISALIGNED and there(pos=A + 2) == MISALIGNED

    def back(d=A, ldd=64, pos=A, add=None, lda=0, dx=A, ldx=64, T=4, D=64, k=2, n=8, type=0, atype=0):
        return L.swiglu_moe_dispatch_bwd(d, ldd, pos, add, lda, dx, ldx, T, D, k, n, type, atype, None)

    assert back(T=0) == 0 and back(d=None) == INVALID and back(dx=None) == INVALID
    assert back(add=A, lda=63) == INVALID and back(add=A, lda=64, atype=1) == INVALID and back(add=A + 2, lda=64, atype=2) == MISALIGNED

    def combine(rows=A, ldr=64, pos=A, gates=A, res=None, ldres=0, y=A, ldy=64, T=4, D=64, k=2, n=8, type=0, p=0.5, step=None):
        return L.swiglu_moe_combine_fwd(rows, ldr, pos, gates, res, ldres, y, ldy, T, D, k, n, type, p, 1, 2, step, None)

    assert combine(T=0) == 0 and combine(p=-0.1) == INVALID and combine(p=1.1) == INVALID and combine(p=float("nan")) == INVALID
    assert combine(T=0, p=2.0) == INVALID
    assert combine(gates=None) == INVALID and combine(rows=None) == INVALID and combine(res=A, ldres=1) == INVALID
    assert combine(step=A + 4) == MISALIGNED and combine(y=A + 1) == MISALIGNED

    def grad(dy=A, lddy=64, rows=A, ldr=64, pos=A, gates=A, d=A, ldd=64, dg=A, T=4, D=64, k=2, n=8, type=0, p=0.5):
        return L.swiglu_moe_combine_bwd(dy, lddy, rows, ldr, pos, gates, d, ldd, dg, T, D, k, n, type, p, 1, 2, None, None)

    assert grad(T=0) == 0 and grad(dg=None) == INVALID and grad(d=None) == INVALID and grad(p=2.0) == INVALID
    assert grad(lddy=1) == INVALID and grad(ldd=1) == INVALID and grad(dg=A + 2) == MISALIGNED

    def drop(x=A, ldx=64, r=None, ldr=0, y=A, ldy=64, M=4, D=64, type=0, p=0.5, step=None):
        return L.swiglu_mlp_dropout(x, ldx, r, ldr, y, ldy, M, D, type, p, 1, 2, step, None)

    assert drop(M=0) == 0 and drop(M=-1) == INVALID and drop(p=1.5) == INVALID and drop(x=None) == INVALID
    assert drop(r=A, ldr=3) == INVALID and drop(ldy=63) == INVALID and drop(type=4) == INVALID
    assert drop(y=A + 1) == MISALIGNED and drop(step=A + 1) == MISALIGNED
    assert b"dropout" in L.swiglu_mlp_last_error_detail()

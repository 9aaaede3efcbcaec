"""Refusals of the operators around the block (CPU only): the binding checks what it is
given, the C entry points check again, before anything reaches a device."""
import ctypes
import re

import pytest
import torch

from helpers import ensure_library

CUDA = "must live on a CUDA device"
bf, hf, f32 = torch.bfloat16, torch.float16, torch.float32
M, D = 6, 40
A = 0x10000            # fake, aligned addresses: validation never dereferences them
INVALID, SHAPE, MISALIGNED, WS = 1, 2, 3, 4


@pytest.fixture(scope="module")
def b():
    ensure_library()
    from bwd_gemm_epilogue_gb300 import binding
    binding.lib()
    return binding


def z(*shape, dtype=bf, device="cpu"):
    return torch.zeros(*shape, dtype=dtype, device=device)


def test_legal_calls_pass_every_check_but_the_device(b):
    x, w, st = z(M, D), z(D, dtype=f32), z(M, dtype=f32)
    for call in (lambda: b.swiglu_mlp_layer_norm_fwd(x, w, w, residual=x),
                 lambda: b.swiglu_mlp_layer_norm_fwd(x),
                 lambda: b.swiglu_mlp_layer_norm_bwd(x, x, w, st, st, dskip=x),
                 lambda: b.swiglu_mlp_clip_grads([x, w], 1.0),
                 lambda: b.swiglu_mlp_grad_norm([x, w])):
        with pytest.raises(ValueError, match=CUDA):
            call()


def test_wrong_tensors_are_refused_by_name(b):
    x, w, st = z(M, D), z(D, dtype=f32), z(M, dtype=f32)
    fwd, bwd, clip = b.swiglu_mlp_layer_norm_fwd, b.swiglu_mlp_layer_norm_bwd, b.swiglu_mlp_clip_grads
    for call, err, match in [
        (lambda: fwd(z(M, D, dtype=torch.float64)), TypeError, "x: torch.float64"),
        (lambda: fwd(z(2, M, D)), ValueError, "x: shape"),
        (lambda: fwd(x, z(D, dtype=hf)), TypeError, "gamma, beta: torch.float16"),
        (lambda: fwd(x, z(D + 1, dtype=f32)), ValueError, "gamma: shape"),
        (lambda: fwd(x, w, z(D)), TypeError, "beta: torch.bfloat16"),
        (lambda: fwd(x, w, w, residual=z(M, D, dtype=f32)), TypeError, "residual: torch.float32"),
        (lambda: fwd(x, w, w, residual=z(M + 1, D)), ValueError, "residual: shape"),
        (lambda: fwd(x, w, w, s=x), ValueError, "s: only written"),
        (lambda: fwd(x, w, w, y=z(D, M).T), ValueError, "y: each row"),
        (lambda: fwd(z(D, M).T, w, w), ValueError, "x: each row"),
        (lambda: fwd(z(1, D).expand(M, D), w, w), ValueError, "x: each row"),
        (lambda: fwd(x, w, w, mean=z(M)), TypeError, "mean: torch.bfloat16"),
        (lambda: fwd(x, z(2 * D, dtype=f32)[::2]), ValueError, "gamma: must be contiguous"),
        (lambda: bwd(z(M, D + 1), x, w, st, st), ValueError, "dy: shape"),
        (lambda: bwd(x, x, w, z(M + 1, dtype=f32), st), ValueError, "mean: shape"),
        (lambda: bwd(x, x, w, st, st, dgamma=z(D)), TypeError, "dgamma: torch.bfloat16"),
        (lambda: bwd(x, x, w, st, st, dbeta=w, param_grads=False), ValueError, "param_grads"),
        (lambda: clip([], 1.0), ValueError, "grads: empty"),
        (lambda: clip([z(D, M).T], 1.0), ValueError, "must be contiguous"),
        (lambda: clip([z(D, dtype=torch.int32)], 1.0), TypeError, r"grads\[0\]: torch.int32"),
        (lambda: clip([x, w], 1.0, out=[x]), ValueError, "out: one tensor"),
        (lambda: clip([x, w], 1.0, out=[x, x]), ValueError, "out: one tensor"),
    ]:
        with pytest.raises(err, match=match):
            call()


def test_headers_and_binding_agree(b):
    src = re.sub(r"/\*.*?\*/", "", open(ensure_header()).read(), flags=re.S)
    names = set(re.findall(r"\b(swiglu_\w+)\s*\(", src))
    assert len(names) == 5
    for n in names:
        assert hasattr(b.lib(), n) and n in b.SIGNATURES


def ensure_header():
    import os

    from helpers import ROOT
    return os.path.join(ROOT, "include", "swiglu_ops.h")


def test_layer_norm_argument_errors(b):
    L = b.lib()

    def fwd(x=A, ldx=64, r=None, ldr=0, gamma=A, beta=A, y=A, ldy=64, s=None, lds=0, mean=A, rstd=A, M=4, D=64,
            eps=1e-5, type=0, wtype=2):
        return L.swiglu_mlp_layer_norm_fwd(x, ldx, r, ldr, gamma, beta, y, ldy, s, lds, mean, rstd, M, D, eps, type,
                                           wtype, None)

    assert fwd(M=0) == 0                                            # nothing to do
    assert fwd(M=-1) == INVALID and fwd(D=0) == INVALID
    assert fwd(M=1 << 31) == SHAPE
    assert fwd(type=3) == INVALID and fwd(type=0, wtype=1) == INVALID and fwd(type=2, wtype=0) == INVALID
    assert fwd(x=None) == INVALID and fwd(y=None) == INVALID
    assert fwd(r=A, ldr=64) == INVALID and fwd(s=A, lds=64) == INVALID      # residual and s go together
    assert fwd(mean=None) == INVALID
    assert fwd(ldx=63) == INVALID and fwd(ldy=0) == INVALID
    assert fwd(eps=-1.0) == INVALID and fwd(eps=float("nan")) == INVALID
    assert fwd(x=A + 1) == MISALIGNED and fwd(gamma=A + 2) == MISALIGNED and fwd(mean=A + 2) == MISALIGNED
    assert b"layer norm" in L.swiglu_mlp_last_error_detail()

    def bwd(dy=A, s=A, gamma=A, mean=A, rstd=A, skip=None, ldk=0, dx=A, dg=A, db=A, M=4, D=64, type=0, wtype=2, ws=A,
            wsb=1 << 40, ld=64):
        return L.swiglu_mlp_layer_norm_bwd(dy, ld, s, ld, gamma, mean, rstd, skip, ldk, dx, ld, dg, db, M, D, type,
                                           wtype, ws, wsb, None)

    assert bwd(M=-1) == INVALID and bwd(type=7) == INVALID
    assert bwd(dy=None) == INVALID and bwd(rstd=None) == INVALID and bwd(ws=None) == INVALID
    assert bwd(ld=60) == INVALID and bwd(skip=A, ldk=1) == INVALID
    assert bwd(ws=A + 8) == MISALIGNED and bwd(dg=A + 2) == MISALIGNED and bwd(dx=A + 1) == MISALIGNED
    need = b.swiglu_mlp_layer_norm_bwd_workspace_size(4, 64)
    assert need > 0 and bwd(wsb=need - 1) == WS
    assert b.swiglu_mlp_layer_norm_bwd_workspace_size(0, 64) == 0


def test_clip_argument_errors(b):
    L = b.lib()

    def clip(ptrs=(A, A), outs=(A, A), counts=(5, 6), types=(0, 2), n=2, max_norm=1.0, eps=1e-6, norm=A, ws=A,
             wsb=1 << 20):
        p = (ctypes.c_void_p * 2)(*ptrs)
        o = None if outs is None else (ctypes.c_void_p * 2)(*outs)
        return L.swiglu_mlp_clip_grads(p, o, (ctypes.c_int64 * 2)(*counts), (ctypes.c_int * 2)(*types), n, max_norm,
                                       eps, norm, ws, wsb, None)

    assert clip(n=-1) == INVALID
    assert clip(outs=None, norm=None) == INVALID
    assert clip(ws=None) == INVALID and clip(ws=A + 4) == MISALIGNED and clip(wsb=8) == WS
    assert clip(ptrs=(A, None)) == INVALID and clip(outs=(None, A)) == INVALID
    assert clip(counts=(5, -1)) == INVALID and clip(types=(0, 3)) == INVALID
    assert clip(ptrs=(A + 1, A)) == MISALIGNED and clip(ptrs=(A, A + 2)) == MISALIGNED
    assert clip(max_norm=-1.0) == INVALID and clip(max_norm=float("nan")) == INVALID and clip(eps=-1.0) == INVALID
    assert clip(norm=A + 2) == MISALIGNED


def test_routed_layer_refusals(b):
    E, H, Do, k = 5, 24, 32, 2
    x, Wr, W1, W2 = z(M, D), z(E, D), z(E, 2 * H, D), z(E, Do, H)
    f = b.swiglu_moe_routed_fwd
    for call, err, match in [
        (lambda: f(x, Wr, W1, W2, k), ValueError, CUDA),
        (lambda: f(x, Wr.float(), W1, W2, k, residual=z(M, Do)), ValueError, CUDA),
        (lambda: f(x, z(E + 1, D), W1, W2, k), ValueError, "Wr: shape"),
        (lambda: f(x, Wr.half(), W1, W2, k), TypeError, "Wr: torch.float16"),
        (lambda: f(x.float(), Wr, W1, W2, k), TypeError, "x: torch.float32"),
        (lambda: f(x, Wr, W1, z(E, Do, H + 8), k), ValueError, "shape mismatch"),
        (lambda: f(x, Wr, W1, W2, k, residual=z(M, D)), ValueError, "residual: shape"),
        (lambda: f(x, Wr, W1, W2, k, y=z(M, D)), ValueError, "y: shape"),
        (lambda: f(x, Wr, W1, W2, k, ids=z(M, k, dtype=torch.int64)), TypeError, "ids: torch.int64"),
        (lambda: f(x, Wr, W1, W2, k, gates=z(M, k)), TypeError, "gates: torch.bfloat16"),
        (lambda: f(x, z(D, E).T, W1, W2, k), ValueError, "Wr: must be contiguous"),
    ]:
        with pytest.raises(err, match=match):
            call()

    L = b.lib()

    def call(x=A, wr=A, r=None, y=A, ids=A, gates=A, T=4, E=8, D=64, H=64, Do=64, k=2, ws=A, wsb=1 << 30):
        return L.swiglu_moe_routed_fwd(x, wr, A, A, r, y, ids, gates, T, E, D, H, Do, k, 1, 0, ws, wsb, None)

    assert call(T=0) == 0
    assert call(T=-1) == INVALID and call(k=0) == INVALID and call(k=9) == INVALID and call(E=0) == INVALID
    assert call(T=65) == SHAPE and call(E=683) == SHAPE and call(E=64, k=17) == SHAPE and call(D=60) == SHAPE
    assert call(H=1 << 24) == SHAPE
    assert call(x=None) == INVALID and call(gates=None) == INVALID and call(ws=None) == INVALID
    assert call(wr=A + 8) == MISALIGNED and call(r=A + 2) == MISALIGNED and call(ids=A + 2) == MISALIGNED
    need = b.swiglu_moe_routed_fwd_workspace_size(4, 64, 64, 2)
    assert need > 4 * 2 * 64 * 2 and call(wsb=need - 1) == WS
    assert b.swiglu_moe_routed_fwd_workspace_size(0, 64, 64, 2) == 0


def test_tensors_on_another_device_than_the_current_one_are_refused(b, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError, match="current CUDA device"):
        b._device_stream(torch.device("cuda", 0))

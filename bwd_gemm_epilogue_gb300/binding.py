"""ctypes binding of the C ABI in ``include/swiglu_mlp.h``, ``include/swiglu_moe.h`` and
``include/swiglu_ops.h`` -- argument marshalling only.

Each function has the name of the C entry point it calls and takes torch CUDA
tensors for the pointer arguments (bf16, contiguous; the operators of
``swiglu_ops.h`` also take fp16 and fp32, and rows at a stride); torch supplies device
memory and the current stream, every step of the computation runs in the
library's kernels.  Outputs and workspaces the caller does not pass are
allocated with torch.  A non-OK status raises ``SwigluError``; a missing
library raises ``RuntimeError`` (there is no fallback path).
"""
from __future__ import annotations

import ctypes
import importlib
import operator
import os
import struct
import threading
import warnings

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libswiglu_mlp.so")

STATUS_NAMES = {
    0: "SWIGLU_OK",
    1: "SWIGLU_ERR_INVALID_ARG",
    2: "SWIGLU_ERR_UNSUPPORTED_SHAPE",
    3: "SWIGLU_ERR_MISALIGNED",
    4: "SWIGLU_ERR_WORKSPACE_TOO_SMALL",
    5: "SWIGLU_ERR_LAUNCH",
    6: "SWIGLU_ERR_TIMEOUT",
    7: "SWIGLU_ERR_CUDA",
}

# Every symbol the headers under include/ declare: name -> (restype, argtypes)
_f32 = ctypes.c_float
_vp, _i64, _i32, _u64, _sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_uint64, ctypes.c_size_t
SIGNATURES = {
    "swiglu_mlp_fwd_workspace_size": (_sz, [_i64, _i64, _i64, _i64]),
    "swiglu_mlp_bwd_workspace_size": (_sz, [_i64, _i64, _i64, _i64]),
    "swiglu_mlp_fwd": (_i32, [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _vp, _sz, _vp]),
    "swiglu_mlp_bwd": (_i32, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _vp, _sz, _vp]),
    "swiglu_mlp_fwd_residual": (_i32, [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _vp, _sz, _vp]),
    "swiglu_mlp_bwd_residual": (_i32, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _vp, _sz, _vp]),
    "swiglu_mlp_fwd_noalloc": (_i32, [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _vp]),
    "swiglu_mlp_fwd_fp8_workspace_size": (_sz, [_i64, _i64, _i64, _i64]),
    "swiglu_mlp_fwd_fp8": (_i32, [_vp, _vp, _vp, ctypes.c_float, ctypes.c_float, ctypes.c_float, ctypes.c_float,
                                  _vp, _vp, _vp, _i64, _i64, _i64, _i64, _vp, _sz, _vp]),
    "swiglu_mlp_fused_grad_preact": (_i32, [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp]),
    "swiglu_mlp_gemm_bf16": (_i32, [_vp, _vp, _vp, _i64, _i64, _i64, _i32, _i32, _vp]),
    "swiglu_mlp_device_status": (_i32, [_vp]),
    "swiglu_mlp_strerror": (ctypes.c_char_p, [_i32]),
    "swiglu_mlp_last_error_detail": (ctypes.c_char_p, []),
    "swiglu_mlp_set_wait_timeout_ns": (None, [_u64]),
    "swiglu_mlp_set_debug_flags": (None, [_i32]),
    "swiglu_mlp_set_raster_band": (None, [_i32]),
    "swiglu_mlp_split_plan": (_i32, [_i64, _i64, _i64, _i32, _vp, _i32]),
    "swiglu_mlp_trace_begin": (None, [_vp, _vp, _i32]),
    "swiglu_mlp_trace_end": (_i32, []),
    "swiglu_mlp_abi_version": (_i32, []),
    "swiglu_mlp_tp_shard_pack": (_i32, [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _i64, _vp]),
    "swiglu_mlp_tp_shard_unpack_grads": (_i32, [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _i64, _vp]),
    "swiglu_mlp_tp_fwd": (_i32, [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _i32, _vp, _vp, _sz, _vp]),
    "swiglu_mlp_tp_chunk_rows": (_i64, [_i64, _i32]),
    "swiglu_mlp_tp_bwd": (_i32, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _vp, _vp, _sz,
                                 _vp]),
    "swiglu_moe_fwd_workspace_size": (_sz, [_vp, _i64, _i64, _i64, _i64]),
    "swiglu_moe_bwd_workspace_size": (_sz, [_vp, _i64, _i64, _i64, _i64]),
    "swiglu_moe_fwd": (_i32, [_vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _vp, _sz, _vp]),
    "swiglu_moe_bwd": (_i32, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _vp, _sz,
                              _vp]),
    "swiglu_moe_routed_fwd_workspace_size": (_sz, [_i64, _i64, _i64, _i64]),
    "swiglu_moe_routed_fwd": (_i32, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _i64, _i64, _i32,
                                     _i32, _vp, _sz, _vp]),
    "swiglu_mlp_layer_norm_fwd": (_i32, [_vp, _i64, _vp, _i64, _vp, _vp, _vp, _i64, _vp, _i64, _vp, _vp, _i64, _i64,
                                         _f32, _i32, _i32, _vp]),
    "swiglu_mlp_layer_norm_bwd_workspace_size": (_sz, [_i64, _i64]),
    "swiglu_mlp_layer_norm_bwd": (_i32, [_vp, _i64, _vp, _i64, _vp, _vp, _vp, _vp, _i64, _vp, _i64, _vp, _vp, _i64,
                                         _i64, _i32, _i32, _vp, _sz, _vp]),
    "swiglu_mlp_clip_grads_workspace_size": (_sz, [_i64]),
    "swiglu_mlp_clip_grads": (_i32, [_vp, _vp, _vp, _vp, _i64, _f32, _f32, _vp, _vp, _sz, _vp]),
}

KERNEL_KINDS = {1: "fwd_preact", 2: "fwd_down", 3: "bwd_grad_h", 4: "bwd_dW2", 5: "bwd_dx", 6: "bwd_dW1", 7: "gemm",
                8: "bwd_gemms", 9: "elementwise", 10: "norm_fwd", 11: "norm_bwd", 12: "norm_params", 13: "grad_norm",
                14: "grad_scale", 15: "moe_route", 16: "moe_up", 17: "moe_down", 18: "moe_join"}


class SwigluError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str = ""):
        self.status = status
        self.detail = detail
        msg = f"{where}: {STATUS_NAMES.get(status, status)}"
        super().__init__(f"{msg} ({detail})" if detail else msg)


_lock = threading.Lock()
_lib = None


def lib() -> ctypes.CDLL:
    """The loaded C library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    f"{LIB_PATH} is missing: build the CUDA library first "
                    "(python -c 'import __graft_entry__ as g; g.build()')")
            handle = ctypes.CDLL(LIB_PATH)
            for name, (res, args) in SIGNATURES.items():
                fn = getattr(handle, name)
                fn.restype = res
                fn.argtypes = args
            _lib = handle
    return _lib


def _check(status: int, where: str) -> None:
    if status != 0:
        raise SwigluError(status, where, lib().swiglu_mlp_last_error_detail().decode(errors="replace"))


def _ptr(t: torch.Tensor | None):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensor must live on a CUDA device")
    if t.dtype not in (torch.bfloat16, torch.uint8, torch.float8_e4m3fn):
        raise TypeError(f"expected bf16, FP8 E4M3 (or a uint8 workspace), got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(device) -> ctypes.c_void_p:
    """The current stream of `device`, which must be the current CUDA device: the
    library launches on the current device (and keeps its per-device state there),
    so tensors on another GPU would be addressed from the wrong one."""
    if device is not None:
        device = torch.device(device)
        if device.type == "cuda" and device.index is not None and device.index != torch.cuda.current_device():
            raise ValueError(f"tensors are on {device} but the current CUDA device is cuda:"
                             f"{torch.cuda.current_device()}; call inside torch.cuda.device({device.index})")
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _empty(shape, like: torch.Tensor) -> torch.Tensor:
    return torch.empty(shape, dtype=torch.bfloat16, device=like.device)


# The kernels' tensor maps are built from the sizes, not from the tensors: a buffer of the
# wrong shape would be read or written past its end.  So every tensor a call receives is
# checked against the shape, dtype and device the sizes imply, before anything is launched.

def _expect(t: torch.Tensor, name: str, shape, dtype, device) -> torch.Tensor:
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name}: {t.dtype}, expected {dtype}")
    if t.device != device:
        raise ValueError(f"{name}: on {t.device}, the call's other tensors are on {device}")
    return t


def _out(t, name: str, shape, like: torch.Tensor, dtype=torch.bfloat16) -> torch.Tensor:
    """A caller's output buffer, checked, or a new one."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    return _expect(t, name, shape, dtype, like.device)


def _same_device(like: torch.Tensor, **tensors) -> None:
    for name, t in tensors.items():
        if t is not None and t.device != like.device:
            raise ValueError(f"{name}: on {t.device}, the call's other tensors are on {like.device}")


def _nbytes(t) -> int:
    return 0 if t is None else t.numel() * t.element_size()


# ---------------------------------------------------------------------------- sizes / status

def swiglu_mlp_fwd_workspace_size(M: int, D: int, H: int, Dout: int) -> int:
    return int(lib().swiglu_mlp_fwd_workspace_size(M, D, H, Dout))


def swiglu_mlp_bwd_workspace_size(M: int, D: int, H: int, Dout: int) -> int:
    return int(lib().swiglu_mlp_bwd_workspace_size(M, D, H, Dout))


def swiglu_mlp_strerror(status: int) -> str:
    return lib().swiglu_mlp_strerror(status).decode()


def swiglu_mlp_device_status(device=None) -> int:
    """Synchronise the current stream and return the device status code (0 = OK)."""
    return int(lib().swiglu_mlp_device_status(_stream(device)))


def swiglu_mlp_set_wait_timeout_ns(ns: int) -> None:
    lib().swiglu_mlp_set_wait_timeout_ns(int(ns))


def swiglu_mlp_set_debug_flags(flags: int) -> None:
    lib().swiglu_mlp_set_debug_flags(int(flags))


def swiglu_mlp_set_raster_band(n_tiles: int) -> None:
    lib().swiglu_mlp_set_raster_band(int(n_tiles))


def swiglu_mlp_split_plan(M: int, N: int, K: int, units: int):
    """Tile lists of the down projection with split tiles (host only): a list of
    (pair, tile, first k-block, end k-block, split index or -1), or None where the
    forward splits no tiles for this shape."""
    n = int(lib().swiglu_mlp_split_plan(int(M), int(N), int(K), int(units), None, 0))
    if n < 0:
        return None
    buf = (ctypes.c_int32 * (5 * max(n, 1)))()
    lib().swiglu_mlp_split_plan(int(M), int(N), int(K), int(units), ctypes.cast(buf, ctypes.c_void_p), n)
    return [tuple(buf[5 * i:5 * i + 5]) for i in range(n)]


def swiglu_mlp_abi_version() -> int:
    return int(lib().swiglu_mlp_abi_version())


class LaunchTrace:
    """Brackets every kernel launch of the library (from this thread) with CUDA
    events, for per-kernel timing inside larger calls:

        with LaunchTrace(capacity) as tr:
            ...calls...
        tr.records()  ->  [(kind_name, milliseconds), ...] in launch order
    """

    def __init__(self, capacity: int):
        self.capacity = int(capacity)
        self.events = [torch.cuda.Event(enable_timing=True) for _ in range(2 * self.capacity)]
        for e in self.events:          # torch creates the CUDA event lazily, on first record
            e.record()
        torch.cuda.synchronize()
        self._handles = (ctypes.c_void_p * len(self.events))(*[e.cuda_event for e in self.events])
        self._kinds = (ctypes.c_int * self.capacity)()
        self.count = 0

    def __enter__(self):
        lib().swiglu_mlp_trace_begin(ctypes.cast(self._handles, ctypes.c_void_p),
                                     ctypes.cast(self._kinds, ctypes.c_void_p), self.capacity)
        return self

    def __exit__(self, *exc):
        self.count = int(lib().swiglu_mlp_trace_end())
        return False

    def records(self):
        torch.cuda.synchronize()
        n = min(self.count, self.capacity)
        return [(KERNEL_KINDS.get(self._kinds[i], str(self._kinds[i])),
                 self.events[2 * i].elapsed_time(self.events[2 * i + 1])) for i in range(n)]


# ---------------------------------------------------------------------------- compute

def _dims(x, W1, W2, dtype=torch.bfloat16):
    M, D = x.shape
    H2, D1 = W1.shape
    Dout, H = W2.shape
    if D1 != D or H2 != 2 * H:
        raise ValueError(f"shape mismatch: x {tuple(x.shape)}, W1 {tuple(W1.shape)}, W2 {tuple(W2.shape)}")
    for name, t in (("x", x), ("W1", W1), ("W2", W2)):
        _expect(t, name, t.shape, dtype, x.device)
    return M, D, H, Dout


def swiglu_mlp_fwd(x, W1, W2, preact=None, y=None, workspace=None, residual: bool = False):
    """Forward; returns (preact [M,2H], y [M,Dout]).  residual: y = x + MLP(x)
    (swiglu_mlp_fwd_residual; D == Dout)."""
    M, D, H, Dout = _dims(x, W1, W2)
    preact = _out(preact, "preact", (M, 2 * H), x)
    y = _out(y, "y", (M, Dout), x)
    _same_device(x, workspace=workspace)
    need = swiglu_mlp_fwd_workspace_size(M, D, H, Dout)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=x.device)
    fn = lib().swiglu_mlp_fwd_residual if residual else lib().swiglu_mlp_fwd
    st = fn(_ptr(x), _ptr(W1), _ptr(W2), _ptr(preact), _ptr(y), M, D, H, Dout,
            _ptr(workspace), _nbytes(workspace), _stream(x.device))
    _check(st, "swiglu_mlp_fwd_residual" if residual else "swiglu_mlp_fwd")
    return preact, y


NOALLOC_SCRATCH_BYTES = 64 * 1024 * 1024


def swiglu_mlp_fwd_noalloc(x, W1, W2, preact=None, y=None):
    """Forward whose transient h lives in the library's built-in 64 MiB device array
    instead of a caller workspace (for callers that cannot allocate; M*H <= 2^25).
    Calls share that array: calls that overlap on the GPU race.  Returns (preact, y)."""
    M, D, H, Dout = _dims(x, W1, W2)
    preact = _out(preact, "preact", (M, 2 * H), x)
    y = _out(y, "y", (M, Dout), x)
    st = lib().swiglu_mlp_fwd_noalloc(_ptr(x), _ptr(W1), _ptr(W2), _ptr(preact), _ptr(y), M, D, H, Dout,
                                      _stream(x.device))
    _check(st, "swiglu_mlp_fwd_noalloc")
    return preact, y


def swiglu_mlp_bwd(x, W1, W2, preact, dy, dx=None, dW1=None, dW2=None, workspace=None, residual: bool = False):
    """Backward; returns (dx [M,D], dW1 [2H,D], dW2 [Dout,H]).  residual: dx += dy
    (swiglu_mlp_bwd_residual; D == Dout)."""
    M, D, H, Dout = _dims(x, W1, W2)
    _expect(preact, "preact", (M, 2 * H), torch.bfloat16, x.device)
    _expect(dy, "dy", (M, Dout), torch.bfloat16, x.device)
    dx = _out(dx, "dx", (M, D), x)
    dW1 = _out(dW1, "dW1", (2 * H, D), x)
    dW2 = _out(dW2, "dW2", (Dout, H), x)
    _same_device(x, workspace=workspace)
    need = swiglu_mlp_bwd_workspace_size(M, D, H, Dout)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=x.device)
    fn = lib().swiglu_mlp_bwd_residual if residual else lib().swiglu_mlp_bwd
    st = fn(_ptr(x), _ptr(W1), _ptr(W2), _ptr(preact), _ptr(dy), _ptr(dx), _ptr(dW1), _ptr(dW2),
            M, D, H, Dout, _ptr(workspace), _nbytes(workspace), _stream(x.device))
    _check(st, "swiglu_mlp_bwd_residual" if residual else "swiglu_mlp_bwd")
    return dx, dW1, dW2


# ---------------------------------------------------------------------------- tensor-parallel shards

def swiglu_mlp_tp_shard_pack(W1, W2, j0: int, Hs: int, W1_shard=None, W2_shard=None):
    """Rank shard of the full weights: W1_shard [2*Hs, D] (rows j0.. and H + j0..),
    W2_shard [Dout, Hs] (columns j0..)."""
    H2, D = W1.shape
    Dout, H = W2.shape
    if H2 != 2 * H:
        raise ValueError(f"shape mismatch: W1 {tuple(W1.shape)}, W2 {tuple(W2.shape)}")
    _expect(W1, "W1", (2 * H, D), torch.bfloat16, W1.device)
    _expect(W2, "W2", (Dout, H), torch.bfloat16, W1.device)
    W1_shard = _out(W1_shard, "W1_shard", (2 * Hs, D), W1)
    W2_shard = _out(W2_shard, "W2_shard", (Dout, Hs), W1)
    st = lib().swiglu_mlp_tp_shard_pack(_ptr(W1), _ptr(W2), _ptr(W1_shard), _ptr(W2_shard), D, H, Dout, j0, Hs,
                                        _stream(W1.device))
    _check(st, "swiglu_mlp_tp_shard_pack")
    return W1_shard, W2_shard


def swiglu_mlp_tp_shard_unpack_grads(dW1_shard, dW2_shard, dW1, dW2, j0: int):
    """Write a shard's weight gradients into rows j0.., H + j0.. of dW1 and columns j0.. of dW2."""
    H2, D = dW1.shape
    Dout, H = dW2.shape
    Hs = dW2_shard.shape[1]
    _expect(dW1, "dW1", (2 * H, D), torch.bfloat16, dW1.device)
    _expect(dW2, "dW2", (Dout, H), torch.bfloat16, dW1.device)
    _expect(dW1_shard, "dW1_shard", (2 * Hs, D), torch.bfloat16, dW1.device)
    _expect(dW2_shard, "dW2_shard", (Dout, Hs), torch.bfloat16, dW1.device)
    st = lib().swiglu_mlp_tp_shard_unpack_grads(_ptr(dW1_shard), _ptr(dW2_shard), _ptr(dW1), _ptr(dW2), D, H, Dout,
                                                j0, Hs, _stream(dW1.device))
    _check(st, "swiglu_mlp_tp_shard_unpack_grads")
    return dW1, dW2


def swiglu_mlp_tp_chunk_rows(M: int, n_chunks: int) -> int:
    return int(lib().swiglu_mlp_tp_chunk_rows(M, n_chunks))


def _events(events):
    if not events:
        return None, None
    arr = (ctypes.c_void_p * len(events))(*[ctypes.c_void_p(e.cuda_event) for e in events])
    return arr, len(events)


def swiglu_mlp_tp_fwd(x, W1_shard, W2_shard, preact=None, y=None, workspace=None, n_chunks: int = 1,
                      chunk_events=None):
    """Shard forward: (preact_shard [M, 2*Hs], partial y [M, Dout]).  chunk_events: n_chunks
    torch.cuda.Event objects, recorded when the rows of chunk c of y are final."""
    M, D, Hs, Dout = _dims(x, W1_shard, W2_shard)
    preact = _out(preact, "preact", (M, 2 * Hs), x)
    y = _out(y, "y", (M, Dout), x)
    _same_device(x, workspace=workspace)
    if workspace is None:
        workspace = torch.empty(max(16, swiglu_mlp_fwd_workspace_size(M, D, Hs, Dout)), dtype=torch.uint8,
                                device=x.device)
    if chunk_events is not None and len(chunk_events) != n_chunks:
        raise ValueError(f"chunk_events: {len(chunk_events)} events for {n_chunks} chunks")
    for e in chunk_events or ():
        if e.cuda_event == 0:   # a torch event is created on its first record
            e.record(torch.cuda.current_stream(x.device))
    arr, _ = _events(chunk_events)
    st = lib().swiglu_mlp_tp_fwd(_ptr(x), _ptr(W1_shard), _ptr(W2_shard), _ptr(preact), _ptr(y), M, D, Hs, Dout,
                                 n_chunks, arr, _ptr(workspace), _nbytes(workspace), _stream(x.device))
    _check(st, "swiglu_mlp_tp_fwd")
    return preact, y


def swiglu_mlp_tp_bwd(x, W1_shard, W2_shard, preact, dy, dx=None, dW1=None, dW2=None, workspace=None,
                      dx_event=None):
    """Shard backward: (partial dx [M, D], dW1_shard [2*Hs, D], dW2_shard [Dout, Hs]).
    dx_event: a torch.cuda.Event recorded when dx is final, before the weight gradients."""
    M, D, Hs, Dout = _dims(x, W1_shard, W2_shard)
    _expect(preact, "preact", (M, 2 * Hs), torch.bfloat16, x.device)
    _expect(dy, "dy", (M, Dout), torch.bfloat16, x.device)
    dx = _out(dx, "dx", (M, D), x)
    dW1 = _out(dW1, "dW1", (2 * Hs, D), x)
    dW2 = _out(dW2, "dW2", (Dout, Hs), x)
    _same_device(x, workspace=workspace)
    if workspace is None:
        workspace = torch.empty(max(16, swiglu_mlp_bwd_workspace_size(M, D, Hs, Dout)), dtype=torch.uint8,
                                device=x.device)
    ev = None
    if dx_event is not None:
        if dx_event.cuda_event == 0:
            dx_event.record(torch.cuda.current_stream(x.device))
        ev = ctypes.c_void_p(dx_event.cuda_event)
    st = lib().swiglu_mlp_tp_bwd(_ptr(x), _ptr(W1_shard), _ptr(W2_shard), _ptr(preact), _ptr(dy), _ptr(dx),
                                 _ptr(dW1), _ptr(dW2), M, D, Hs, Dout, ev, _ptr(workspace), _nbytes(workspace),
                                 _stream(x.device))
    _check(st, "swiglu_mlp_tp_bwd")
    return dx, dW1, dW2


def bwd_workspace_views(workspace: torch.Tensor, M: int, H: int):
    """(h [M,H], grad_preact [M,2H]) views of a backward workspace."""
    off = ((M * H * 2) + 255) // 256 * 256
    h = workspace[: M * H * 2].view(torch.bfloat16).view(M, H)
    gp = workspace[off: off + M * 2 * H * 2].view(torch.bfloat16).view(M, 2 * H)
    return h, gp


def swiglu_mlp_fwd_fp8_workspace_size(M: int, D: int, H: int, Dout: int) -> int:
    return int(lib().swiglu_mlp_fwd_fp8_workspace_size(M, D, H, Dout))


def swiglu_mlp_fwd_fp8(x8, W1_8, W2_8, s_x: float, s_w1: float, s_w2: float, s_h: float,
                       preact=None, h8=None, y=None, store_preact: bool = True, workspace=None):
    """FP8 forward (E4M3 operands, per-tensor scales); returns (preact [M,2H] bf16 or
    None, h8 [M,H] E4M3, y [M,Dout] bf16)."""
    M, D, H, Dout = _dims(x8, W1_8, W2_8, dtype=torch.float8_e4m3fn)
    if store_preact:
        preact = _out(preact, "preact", (M, 2 * H), x8)
    h8 = _out(h8, "h8", (M, H), x8, dtype=torch.float8_e4m3fn)
    y = _out(y, "y", (M, Dout), x8)
    _same_device(x8, workspace=workspace)
    if workspace is None:
        n = swiglu_mlp_fwd_fp8_workspace_size(M, D, H, Dout)
        workspace = torch.empty(n, dtype=torch.uint8, device=x8.device) if n else None
    st = lib().swiglu_mlp_fwd_fp8(_ptr(x8), _ptr(W1_8), _ptr(W2_8), s_x, s_w1, s_w2, s_h,
                                  _ptr(preact) if store_preact else None, _ptr(h8), _ptr(y), M, D, H, Dout,
                                  _ptr(workspace), _nbytes(workspace), _stream(x8.device))
    _check(st, "swiglu_mlp_fwd_fp8")
    return (preact if store_preact else None), h8, y


def swiglu_mlp_fused_grad_preact(dy, W2, preact, grad_preact=None, h=None):
    """The fused grad_h GEMM + SwiGLU backward alone; returns (grad_preact [M,2H], h [M,H])."""
    M, Dout = dy.shape
    Dout2, H = W2.shape
    if Dout2 != Dout or tuple(preact.shape) != (M, 2 * H):
        raise ValueError("shape mismatch")
    for name, t in (("dy", dy), ("W2", W2), ("preact", preact)):
        _expect(t, name, t.shape, torch.bfloat16, dy.device)
    grad_preact = _out(grad_preact, "grad_preact", (M, 2 * H), dy)
    h = _out(h, "h", (M, H), dy)
    st = lib().swiglu_mlp_fused_grad_preact(_ptr(dy), _ptr(W2), _ptr(preact), _ptr(grad_preact), _ptr(h),
                                            M, H, Dout, _stream(dy.device))
    _check(st, "swiglu_mlp_fused_grad_preact")
    return grad_preact, h


def swiglu_mlp_gemm_bf16(A, B, M: int, N: int, K: int, a_mn_major: bool, b_mn_major: bool, C=None):
    """C [M,N] = A * B^T; A is [M,K] (or [K,M] if a_mn_major), B is [N,K] (or [K,N] if b_mn_major)."""
    _expect(A, "A", (K, M) if a_mn_major else (M, K), torch.bfloat16, A.device)
    _expect(B, "B", (K, N) if b_mn_major else (N, K), torch.bfloat16, A.device)
    C = _out(C, "C", (M, N), A)
    st = lib().swiglu_mlp_gemm_bf16(_ptr(A), _ptr(B), _ptr(C), M, N, K, int(a_mn_major), int(b_mn_major),
                                    _stream(A.device))
    _check(st, "swiglu_mlp_gemm_bf16")
    return C


class _NoSecondDerivative(torch.autograd.Function):
    """A backward kernel's results (the first n tensors), as functions of all that they were computed
    from (the rest): to differentiate them again raises, where it would else lose their terms."""

    @staticmethod
    def forward(ctx, n, *tensors):
        return tuple(t.view_as(t) for t in tensors[:n])

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError("the backward kernels are not differentiable: no second derivative passes through them")


def _once(outputs, *inputs):
    """A backward's outputs (None among them), guarded when a graph of it is wanted (create_graph)."""
    if not torch.is_grad_enabled():
        return outputs
    own = [t for t in outputs if t is not None]
    guarded = iter(_NoSecondDerivative.apply(len(own), *own, *(t for t in inputs if t is not None)))
    return tuple(None if t is None else next(guarded) for t in outputs)


class SwiGLUMLP(torch.autograd.Function):
    """autograd wrapper: forward saves (x, W1, W2, preact) and drops h; backward
    calls swiglu_mlp_bwd.  Leading dimensions of x are flattened.  With residual
    set it is the block y = x + MLP(x) (the residual entry points).  Differentiable once."""

    @staticmethod
    def forward(ctx, x, W1, W2, residual=False):
        x2 = x.reshape(-1, x.shape[-1]).contiguous()
        preact, y = swiglu_mlp_fwd(x2, W1.contiguous(), W2.contiguous(), residual=residual)
        ctx.save_for_backward(x, W1, W2, preact)
        ctx.residual = residual
        return y.reshape(*x.shape[:-1], y.shape[-1])

    @staticmethod
    def backward(ctx, grad_y):
        x, W1, W2, preact = ctx.saved_tensors
        with torch.no_grad():
            x2 = x.reshape(-1, x.shape[-1]).contiguous()
            dy = grad_y.reshape(-1, grad_y.shape[-1]).contiguous()
            dx, dW1, dW2 = swiglu_mlp_bwd(x2, W1.contiguous(), W2.contiguous(), preact, dy, residual=ctx.residual)
            dx = dx.reshape(*grad_y.shape[:-1], dx.shape[-1])
        return *_once((dx, dW1, dW2), grad_y, x, W1, W2), None


def swiglu_mlp(x, W1, W2, residual: bool = False):
    return SwiGLUMLP.apply(x, W1, W2, residual)


# ---------------------------------------------------------------------------- mixture of experts

def _counts(counts):
    """Host int64 array of the per-expert row counts (kept alive by the caller's frame)."""
    vals = [int(v) for v in (counts.tolist() if hasattr(counts, "tolist") else counts)]
    return (ctypes.c_int64 * len(vals))(*vals), len(vals), sum(vals)


def _moe_dims(x, W1, W2):
    T, D = x.shape
    E, H2, D1 = W1.shape
    E2, Dout, H = W2.shape
    if D1 != D or H2 != 2 * H or E2 != E:
        raise ValueError(f"shape mismatch: x {tuple(x.shape)}, W1 {tuple(W1.shape)}, W2 {tuple(W2.shape)}")
    for name, t in (("x", x), ("W1", W1), ("W2", W2)):
        _expect(t, name, t.shape, torch.bfloat16, x.device)
    return T, E, D, H, Dout


def swiglu_moe_fwd_workspace_size(counts, D: int, H: int, Dout: int) -> int:
    arr, E, _ = _counts(counts)
    return int(lib().swiglu_moe_fwd_workspace_size(ctypes.cast(arr, _vp), E, D, H, Dout))


def swiglu_moe_bwd_workspace_size(counts, D: int, H: int, Dout: int) -> int:
    arr, E, _ = _counts(counts)
    return int(lib().swiglu_moe_bwd_workspace_size(ctypes.cast(arr, _vp), E, D, H, Dout))


def swiglu_moe_fwd(x, W1, W2, counts, preact=None, y=None, workspace=None):
    """Forward of every expert on its rows (x grouped by expert, counts per expert);
    returns (preact [T,2H], y [T,Dout])."""
    T, E, D, H, Dout = _moe_dims(x, W1, W2)
    arr, En, total = _counts(counts)
    if En != E or total != T:
        raise ValueError(f"counts: {En} experts summing to {total}, expected {E} and {T}")
    preact = _out(preact, "preact", (T, 2 * H), x)
    y = _out(y, "y", (T, Dout), x)
    _same_device(x, workspace=workspace)
    if workspace is None:
        workspace = torch.empty(max(16, swiglu_moe_fwd_workspace_size(counts, D, H, Dout)), dtype=torch.uint8,
                                device=x.device)
    st = lib().swiglu_moe_fwd(_ptr(x), _ptr(W1), _ptr(W2), _ptr(preact), _ptr(y), ctypes.cast(arr, _vp), E, D, H,
                              Dout, _ptr(workspace), _nbytes(workspace), _stream(x.device))
    _check(st, "swiglu_moe_fwd")
    return preact, y


def swiglu_moe_bwd(x, W1, W2, preact, dy, counts, dx=None, dW1=None, dW2=None, workspace=None):
    """Backward of every expert on its rows; returns (dx [T,D], dW1 [E,2H,D], dW2 [E,Dout,H])."""
    T, E, D, H, Dout = _moe_dims(x, W1, W2)
    arr, En, total = _counts(counts)
    if En != E or total != T:
        raise ValueError(f"counts: {En} experts summing to {total}, expected {E} and {T}")
    _expect(preact, "preact", (T, 2 * H), torch.bfloat16, x.device)
    _expect(dy, "dy", (T, Dout), torch.bfloat16, x.device)
    dx = _out(dx, "dx", (T, D), x)
    dW1 = _out(dW1, "dW1", (E, 2 * H, D), x)
    dW2 = _out(dW2, "dW2", (E, Dout, H), x)
    _same_device(x, workspace=workspace)
    if workspace is None:
        workspace = torch.empty(max(16, swiglu_moe_bwd_workspace_size(counts, D, H, Dout)), dtype=torch.uint8,
                                device=x.device)
    st = lib().swiglu_moe_bwd(_ptr(x), _ptr(W1), _ptr(W2), _ptr(preact), _ptr(dy), _ptr(dx), _ptr(dW1),
                              _ptr(dW2), ctypes.cast(arr, _vp), E, D, H, Dout, _ptr(workspace),
                              _nbytes(workspace), _stream(x.device))
    _check(st, "swiglu_moe_bwd")
    return dx, dW1, dW2


def swiglu_moe_routed_fwd_workspace_size(T: int, H: int, Dout: int, top_k: int) -> int:
    return int(lib().swiglu_moe_routed_fwd_workspace_size(T, H, Dout, top_k))


def swiglu_moe_routed_fwd(x, Wr, W1, W2, top_k: int, renormalize: bool = True, residual=None, y=None, ids=None,
                          gates=None, workspace=None):
    """A whole MoE layer for up to 64 tokens, routed on the device: returns (y [T,Dout] bf16,
    ids [T,top_k] int32, gates [T,top_k] fp32).  Wr [E,D] bf16 or fp32; residual [T,Dout] is
    added to y; renormalize: the chosen gates sum to one."""
    if y is None and ids is None and gates is None and workspace is None:
        done = _short().moe_routed_fwd(x, Wr, W1, W2, top_k, renormalize, residual)
        if done is not None:
            return done if done.__class__ is tuple else _check(done, "swiglu_moe_routed_fwd")
    if x.dim() != 2 or W1.dim() != 3 or W2.dim() != 3:
        raise ValueError(f"shape mismatch: x {tuple(x.shape)}, W1 {tuple(W1.shape)}, W2 {tuple(W2.shape)}")
    T, D = x.shape
    E, Dout, H = W2.shape
    bf, device = torch.bfloat16, x.device
    if W1.shape != (E, 2 * H, D):
        raise ValueError(f"shape mismatch: x {tuple(x.shape)}, W1 {tuple(W1.shape)}, W2 {tuple(W2.shape)}")
    fp32 = Wr.dtype == torch.float32
    px, pr = _vector(x, "x", (T, D), bf, device), _vector(Wr, "Wr", (E, D), torch.float32 if fp32 else bf, device)
    p1, p2 = _vector(W1, "W1", W1.shape, bf, device), _vector(W2, "W2", W2.shape, bf, device)
    pres = _vector(residual, "residual", (T, Dout), bf, device)
    y, py = _out_vector(y, "y", (T, Dout), bf, device)
    ids, pids = _out_vector(ids, "ids", (T, top_k), torch.int32, device)
    gates, pgates = _out_vector(gates, "gates", (T, top_k), torch.float32, device)
    need = lib().swiglu_moe_routed_fwd_workspace_size(T, H, Dout, top_k) if workspace is None else 0
    workspace, pw, nw = _workspace(workspace, need, device)
    st = lib().swiglu_moe_routed_fwd(px, pr, p1, p2, pres, py, pids, pgates, T, E, D, H, Dout, top_k,
                                     bool(renormalize), fp32, pw, nw, _device_stream(device))
    if st:
        _check(st, "swiglu_moe_routed_fwd")
    return y, ids, gates


# ---------------------------------------------------------------------------- layer norm

_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}      # swiglu_dtype
_dtype_of = operator.attrgetter("dtype")


# The calls below are short on the device (a few microseconds for a decode step's tokens), so
# the usual ones, every output new, are made by a compiled module (csrc/ops/short_calls.cpp), which
# returns None for any other and for anything unexpected.  Here the checks compare first and
# explain (in _expect) only on a mismatch, and the stream comes from torch's raw accessor.
_short_calls = None


class _NoShortCalls:
    """In the module's place where it was not built or is another torch's: every call is made below."""

    def __getattr__(self, name):
        return lambda *args: None


def _short():
    global _short_calls
    if _short_calls is None:
        lib()                              # says what to do where it has not been built
        try:
            module = importlib.import_module("._short_calls", __package__)
            if module.torch_version != str(torch.__version__):
                raise ImportError(f"it was built for torch {module.torch_version}, not {torch.__version__}")
        except ImportError as e:
            warnings.warn(f"the short operators' calls go through ctypes: {e}")
            module = _NoShortCalls()
        _short_calls = module
    return _short_calls


_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else None


def _device_stream(device) -> int:
    """The current stream of `device`, refused where that is not the current CUDA device."""
    if device.type != "cuda":
        raise ValueError("tensor must live on a CUDA device")
    if _raw_stream is None or device.index != torch.cuda.current_device():
        return _stream(device).value       # raises for another device than the current one
    return _raw_stream(device.index)


def _dtype(t: torch.Tensor, name: str) -> int:
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name}: {t.dtype}, expected bf16, fp16 or fp32")
    return code


def _rows(t, name: str, shape, dtype, device):
    """(pointer, row stride) of a [M, D] tensor whose rows are contiguous; (None, 0) for None."""
    if t is None:
        return None, 0
    if t.shape != shape or t.dtype != dtype or t.device != device:
        _expect(t, name, shape, dtype, device)
    ld, one = t.stride()
    if one != 1 or ld < shape[1]:
        if (one != 1 and shape[1] > 1) or (ld < shape[1] and shape[0] > 1):
            raise ValueError(f"{name}: each row must be contiguous and rows must not overlap (strides {t.stride()})")
        ld = max(ld, shape[1])
    return t.data_ptr(), ld


def _vector(t, name: str, shape, dtype, device):
    """Pointer of a contiguous tensor, or None."""
    if t is None:
        return None
    if t.shape != shape or t.dtype != dtype or t.device != device:
        _expect(t, name, shape, dtype, device)
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    return t.data_ptr()


def _out_rows(t, name: str, shape, dtype, device):
    """(tensor, pointer, row stride) of a [M, D] output: the caller's, checked, or a new one."""
    if t is None:
        t = torch.empty(shape, dtype=dtype, device=device)
        return t, t.data_ptr(), shape[1]
    return (t, *_rows(t, name, shape, dtype, device))


def _out_vector(t, name: str, shape, dtype, device):
    """(tensor, pointer) of a contiguous output: the caller's, checked, or a new one."""
    if t is None:
        t = torch.empty(shape, dtype=dtype, device=device)
        return t, t.data_ptr()
    return t, _vector(t, name, shape, dtype, device)


def _workspace(t, need: int, device):
    """(tensor, pointer, bytes) of a workspace: the caller's, or a new one of `need` bytes."""
    if t is None:
        t = torch.empty(max(16, need), dtype=torch.uint8, device=device)
        return t, t.data_ptr(), max(16, need)
    return t, _workspace_ptr(t, device), _nbytes(t)


def _workspace_ptr(t: torch.Tensor, device):
    if t.device != device:
        raise ValueError(f"workspace: on {t.device}, the call's other tensors are on {device}")
    if not t.is_contiguous():
        raise ValueError("workspace: must be contiguous")
    return t.data_ptr()


def _norm_params(x, gamma, beta):
    """dtype of gamma and beta (x's, where there are none)."""
    wdtype = gamma.dtype if gamma is not None else beta.dtype if beta is not None else x.dtype
    if wdtype != x.dtype and wdtype != torch.float32:
        raise TypeError(f"gamma, beta: {wdtype}, expected {x.dtype} or torch.float32")
    return wdtype


def swiglu_mlp_layer_norm_fwd(x, gamma=None, beta=None, eps: float = 1e-5, residual=None, y=None, s=None, mean=None,
                              rstd=None):
    """Layer norm of x (+ residual); returns (y, s, mean, rstd): s is x + residual, or x itself
    without a residual; mean, rstd [M] fp32 are what the backward takes.  x, residual, y, s
    [M, D] bf16, fp16 or fp32, rows at any stride; gamma, beta [D] of x's type or fp32.  y and s
    may each be x or residual (in place), but not both the same."""
    if y is None and s is None and mean is None and rstd is None:
        done = _short().layer_norm_fwd(x, gamma, beta, eps, residual)
        if done is not None:
            return done if done.__class__ is tuple else _check(done, "swiglu_mlp_layer_norm_fwd")
    if x.dim() != 2:
        raise ValueError(f"x: shape {tuple(x.shape)}, expected two dimensions")
    shape, dtype, device = x.shape, x.dtype, x.device
    M, D = shape
    code, wdtype = _dtype(x, "x"), _norm_params(x, gamma, beta)
    px, ldx = _rows(x, "x", shape, dtype, device)
    pr, ldr = _rows(residual, "residual", shape, dtype, device)
    pgamma, pbeta = _vector(gamma, "gamma", (D,), wdtype, device), _vector(beta, "beta", (D,), wdtype, device)
    y, py, ldy = _out_rows(y, "y", shape, dtype, device)
    ps, lds = None, 0
    if residual is not None:
        s, ps, lds = _out_rows(s, "s", shape, dtype, device)
    elif s is not None:
        raise ValueError("s: only written with a residual")
    mean, pmean = _out_vector(mean, "mean", (M,), torch.float32, device)
    rstd, prstd = _out_vector(rstd, "rstd", (M,), torch.float32, device)
    st = lib().swiglu_mlp_layer_norm_fwd(px, ldx, pr, ldr, pgamma, pbeta, py, ldy, ps, lds, pmean, prstd, M, D, eps,
                                         code, _DTYPES[wdtype], _device_stream(device))
    if st:
        _check(st, "swiglu_mlp_layer_norm_fwd")
    return y, (x if s is None else s), mean, rstd


def swiglu_mlp_layer_norm_bwd_workspace_size(M: int, D: int) -> int:
    return int(lib().swiglu_mlp_layer_norm_bwd_workspace_size(M, D))


def swiglu_mlp_layer_norm_bwd(dy, s, gamma, mean, rstd, dskip=None, dx=None, dgamma=None, dbeta=None, workspace=None,
                              param_grads: bool = True):
    """Backward of the layer norm; returns (dx, dgamma, dbeta).  s: the forward's normalised
    input; dskip: a gradient added to dx (the residual stream's).  gamma None (= 1): dgamma
    and dbeta have the type of the dbeta passed in, or s's.  param_grads False: neither is
    computed and both are None.  dx may be dy, s or dskip (in place)."""
    if dx is None and dgamma is None and dbeta is None and workspace is None and param_grads:
        done = _short().layer_norm_bwd(dy, s, gamma, mean, rstd, dskip)
        if done is not None:
            return done if done.__class__ is tuple else _check(done, "swiglu_mlp_layer_norm_bwd")
    if s.dim() != 2:
        raise ValueError(f"s: shape {tuple(s.shape)}, expected two dimensions")
    shape, dtype, device = s.shape, s.dtype, s.device
    M, D = shape
    code, wdtype = _dtype(s, "s"), _norm_params(s, gamma, dbeta)
    pdy, lddy = _rows(dy, "dy", shape, dtype, device)
    ps, lds = _rows(s, "s", shape, dtype, device)
    pk, ldk = _rows(dskip, "dskip", shape, dtype, device)
    pgamma = _vector(gamma, "gamma", (D,), wdtype, device)
    pmean = _vector(mean, "mean", (M,), torch.float32, device)
    prstd = _vector(rstd, "rstd", (M,), torch.float32, device)
    dx, pdx, lddx = _out_rows(dx, "dx", shape, dtype, device)
    pdgamma = pdbeta = None
    if param_grads:
        dgamma, pdgamma = _out_vector(dgamma, "dgamma", (D,), wdtype, device)
        dbeta, pdbeta = _out_vector(dbeta, "dbeta", (D,), wdtype, device)
    elif dgamma is not None or dbeta is not None:
        raise ValueError("dgamma, dbeta: not computed with param_grads=False")
    need = lib().swiglu_mlp_layer_norm_bwd_workspace_size(M, D) if workspace is None else 0
    workspace, pw, nw = _workspace(workspace, need, device)
    st = lib().swiglu_mlp_layer_norm_bwd(pdy, lddy, ps, lds, pgamma, pmean, prstd, pk, ldk, pdx, lddx, pdgamma, pdbeta,
                                         M, D, code, _DTYPES[wdtype], pw, nw, _device_stream(device))
    if st:
        _check(st, "swiglu_mlp_layer_norm_bwd")
    return dx, dgamma, dbeta


class LayerNorm(torch.autograd.Function):
    """autograd wrapper: y without a residual, (y, s) with one; the gradient reaching s past
    the norm is then added to dx in the backward kernel.  Leading dimensions are flattened.
    Differentiable once."""

    @staticmethod
    def forward(ctx, x, gamma, beta, eps, residual):
        y, s, mean, rstd = swiglu_mlp_layer_norm_fwd(_flat_rows(x), gamma, beta, eps,
                                                     None if residual is None else _flat_rows(residual))
        ctx.residual = None if residual is None else residual.shape
        s = x if residual is None else s.reshape(x.shape)
        ctx.save_for_backward(s, gamma, mean, rstd)
        ctx.beta_dtype = None if beta is None else beta.dtype
        ctx.set_materialize_grads(False)
        return y.reshape(x.shape) if residual is None else (y.reshape(x.shape), s)

    @staticmethod
    def backward(ctx, dy, ds=None):
        s, gamma, mean, rstd = ctx.saved_tensors
        if dy is None:
            return ds, None, None, None, _residual_grad(ds, ctx.residual)
        with torch.no_grad():
            rows = _flat_rows(s)
            dbeta = None if ctx.beta_dtype is None else torch.empty(rows.shape[1], dtype=ctx.beta_dtype, device=s.device)
            want = gamma is not None or dbeta is not None
            dx, dgamma, _ = swiglu_mlp_layer_norm_bwd(_flat_rows(dy), rows, gamma, mean, rstd,
                                                      None if ds is None else _flat_rows(ds), dbeta=dbeta,
                                                      param_grads=want)
            dx = dx.reshape(dy.shape)
        dx, dgamma, dbeta = _once((dx, None if gamma is None else dgamma, dbeta), dy, ds, s, gamma)
        return dx, dgamma, dbeta, None, _residual_grad(dx, ctx.residual)


def _residual_grad(dx, shape):
    """dx for a residual of `shape`, whose leading dimensions may be others than x's: the same tensor,
    which autograd copies where it keeps both, or a copy (a view would be kept as it is, and x's
    gradient and the residual's would share their memory)."""
    if dx is None or shape is None:
        return None
    return dx if dx.shape == shape else dx.reshape(shape).clone()


def _flat_rows(t):
    """[..., D] as [M, D] with contiguous, non-overlapping rows (a copy where the strides forbid it)."""
    t = t.reshape(-1, t.shape[-1])
    return t if t.stride(1) == 1 and t.stride(0) >= t.shape[1] else t.contiguous()


def layer_norm(x, gamma=None, beta=None, eps: float = 1e-5, residual=None):
    """(y, s): the layer norm of s = x + residual, and s (x itself without a residual)."""
    out = LayerNorm.apply(x, gamma, beta, eps, residual)
    return out if residual is not None else (out, x)


# ---------------------------------------------------------------------------- gradient clipping

def swiglu_mlp_clip_grads_workspace_size(n: int) -> int:
    return int(lib().swiglu_mlp_clip_grads_workspace_size(n))


def _grad_lists(tensors, name: str):
    """Device, types, element counts and pointers of contiguous tensors on one device.  A
    model's gradients are many: one pass in C for each property."""
    device, of = tensors[0].device, torch.Tensor
    if len(set(map(of.get_device, tensors))) > 1 or not all(map(of.is_contiguous, tensors)):
        for i, t in enumerate(tensors):
            if t.device != device:
                raise ValueError(f"{name}[{i}]: on {t.device}, the call's other tensors are on {device}")
            if not t.is_contiguous():
                raise ValueError(f"{name}[{i}]: tensor must be contiguous")
    return device, list(map(_dtype_of, tensors)), list(map(of.numel, tensors)), list(map(of.data_ptr, tensors))


def _clip_call(grads, max_norm, eps, out, norm, workspace):
    if not grads:
        raise ValueError("grads: empty")
    if norm is None and workspace is None:
        done = _short().clip_grads(grads, out, max_norm, eps)
        if done is not None:
            return done if done.__class__ is not int else _check(done, "swiglu_mlp_clip_grads")
    n = len(grads)
    device, types, counts, ptrs = _grad_lists(grads, "grads")
    try:
        codes = list(map(_DTYPES.__getitem__, types))
    except KeyError:
        i = next(i for i, t in enumerate(types) if t not in _DTYPES)
        raise TypeError(f"grads[{i}]: {types[i]}, expected bf16, fp16 or fp32") from None
    pack = struct.Struct(f"{n}Q").pack
    ins, outs = pack(*ptrs), None
    if out is grads:
        outs = ins
    elif out is not None:
        odevice, otypes, ocounts, optrs = _grad_lists(out, "out") if out else (None,) * 4
        if odevice != device or ocounts != counts or otypes != types:
            raise ValueError("out: one tensor of the same type, element count and device for each gradient")
        outs = pack(*optrs)
    norm, pnorm = _out_vector(norm, "norm", (), torch.float32, device)
    need = lib().swiglu_mlp_clip_grads_workspace_size(n) if workspace is None else 0
    workspace, pw, nw = _workspace(workspace, need, device)
    st = lib().swiglu_mlp_clip_grads(ins, outs, pack(*counts), struct.pack(f"{n}i", *codes), n, max_norm, eps,
                                     pnorm, pw, nw, _device_stream(device))
    if st:
        _check(st, "swiglu_mlp_clip_grads")
    return norm


def swiglu_mlp_clip_grads(grads, max_norm: float, eps: float = 1e-6, out=None, norm=None, workspace=None):
    """Clip gradients by their global norm; returns (norm, clipped gradients).  The result
    goes to `out` (a list like grads), or into grads themselves when out is None.  norm: fp32
    scalar on the device, of the gradients before clipping (no host synchronisation).  Outputs
    that overlap, such as one gradient listed twice, are refused."""
    grads = list(grads)
    dst = grads if out is None else list(out)
    return _clip_call(grads, float(max_norm), float(eps), dst, norm, workspace), dst


def swiglu_mlp_grad_norm(grads, norm=None, workspace=None):
    """Global norm of gradients alone (swiglu_mlp_clip_grads without outputs)."""
    return _clip_call(list(grads), 0.0, 0.0, None, norm, workspace)

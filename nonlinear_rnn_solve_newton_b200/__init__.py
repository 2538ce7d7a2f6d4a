"""Python binding of libpararnn.so: Newton solves of nonlinear RNNs on a B200.

Argument marshalling only.  Every step of the computation runs in the CUDA
kernels of ``libpararnn.so`` (C ABI in ``include/pararnn.h``); torch provides
device memory (outputs, workspace, the info struct) and the current stream.
There is no CPU fallback: if the library is missing or the tensors are not on a
CUDA device, the calls raise.

Entry points (same names as the C ABI, without the ``pararnn_`` prefix):

* ``scan_diag(A, b, h0=None)``      h_t = A_t h_{t-1} + b_t           [B, L, D]
* ``scan_block2(A, b, x0=None)``    x_t = A_t x_{t-1} + b_t, 2x2 blocks  [B, L, D, 2]
* ``solve_gru(P, a, h0=None, tol=1e-4, max_iters=32)``   ParaGRU Newton solve
* ``solve_lstm(P, a, c0=None, h0=None, tol=1e-4, max_iters=32)``  ParaLSTM Newton solve
* ``solve_gru_backward`` / ``solve_lstm_backward``  gradients through the solution
* ``solve_mhgru(P, U, h0=None)``     multi-head GRU, dense 8x8 recurrence blocks
* ``solve_mhgru_strided(P, U, strides, h0=None)``  the same with a time stride per head
* ``input_projection(x, W, bias=None)``  P = x W^T + bias on the tensor cores
* ``solve_gru_projected(x, W, bias, a, h0=None)``  the projection fused with the
  ParaGRU Newton solve (P never reaches HBM)
* ``scan_linattn(q, k, v, log_decay, s0=None)``  linear attention with one decay per
  head over a prompt;  ``scan_linattn_backward``  its gradients;  ``step_linattn``
  one token
* ``layer_norm(x, weight, bias)`` / ``layer_norm_backward``  layer norm and its gradients
* ``step_gru`` / ``step_lstm``      one decode step;  ``rollout_gru`` / ``rollout_lstm``
  the sequential application on the GPU

The workspace the solves and scans need comes from torch's allocator and is
reused between calls on the same thread, device and stream.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import threading

import torch

from . import build as _build

__all__ = ["scan_diag", "scan_block2", "solve_gru", "solve_lstm", "solve_gru_noalloc", "solve_gru_projected", "solve_mhgru_strided",
           "solve_gru_backward", "solve_lstm_backward", "solve_mhgru", "input_projection",
           "step_gru", "step_lstm", "rollout_gru", "rollout_lstm",
           "scan_linattn", "scan_linattn_backward", "step_linattn",
           "layer_norm", "layer_norm_backward",
           "workspace_size", "probe_rate", "PROBE_MUFU", "PROBE_FMA",
           "SolveInfo", "Options", "PararnnError", "library_path", "load", "MAX_ITERS"]

MAX_ITERS = 127
_HERE = os.path.dirname(os.path.abspath(__file__))
library_path = os.path.join(_HERE, "libpararnn.so")

OP_SCAN_DIAG, OP_SCAN_BLOCK2, OP_GRU, OP_LSTM = 0, 1, 2, 3
OP_GRU_BACKWARD, OP_LSTM_BACKWARD = 4, 5
OP_MHGRU = 6
OP_GRU_PROJECTED = 7
OP_MHGRU_STRIDED = 8
F32, BF16 = 0, 1

_STATUS = {0: "ok", 1: "invalid argument", 2: "unsupported device", 3: "CUDA runtime error",
           4: "device-side wait timed out", 5: "non-finite residual",
           6: "workspace missing, too small or misaligned"}


class PararnnError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = int(status)
        super().__init__(f"{where}: {_STATUS.get(self.status, 'unknown status')} ({self.status})")


class _Info(ctypes.Structure):
    _fields_ = [("iterations", ctypes.c_int32), ("converged", ctypes.c_int32),
                ("status", ctypes.c_int32), ("updates", ctypes.c_int32),
                ("passes", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("max_residual", ctypes.c_float), ("rho", ctypes.c_float * (MAX_ITERS + 1))]


class Options(ctypes.Structure):
    """Tuning and test hooks (see pararnn_options_t)."""
    _fields_ = [("iters_first", ctypes.c_int32), ("iters_next", ctypes.c_int32),
                ("wait_timeout_ns", ctypes.c_int64), ("debug_stall_unit", ctypes.c_int64),
                ("regime", ctypes.c_int32), ("walk_warps", ctypes.c_int32),
                ("walk_width", ctypes.c_int32), ("reserved", ctypes.c_int32)]

    AUTO, LOOKBACK, WALK = 0, 1, 2

    def __init__(self, iters_first=0, iters_next=0, wait_timeout_ns=0, debug_stall_unit=-1,
                 regime=0, walk_warps=0, walk_width=0):
        super().__init__(iters_first, iters_next, wait_timeout_ns, debug_stall_unit, regime,
                         walk_warps, walk_width, 0)


class _LinAttn(ctypes.Structure):
    """Shapes and strides of a linear-attention call (see pararnn_linattn_t)."""
    _fields_ = [("B", ctypes.c_int64), ("L", ctypes.c_int64), ("H", ctypes.c_int32),
                ("Hq", ctypes.c_int32), ("Hk", ctypes.c_int32), ("Hv", ctypes.c_int32),
                ("Dk", ctypes.c_int32), ("Dv", ctypes.c_int32), ("scale", ctypes.c_float),
                ("reserved", ctypes.c_int32), ("q_stride", ctypes.c_int64 * 3),
                ("k_stride", ctypes.c_int64 * 3), ("v_stride", ctypes.c_int64 * 3),
                ("do_stride", ctypes.c_int64 * 3)]


_Stride3 = ctypes.c_int64 * 3

INFO_BYTES = ctypes.sizeof(_Info)

_lock = threading.Lock()
_lib = None
_vp = ctypes.c_void_p
_i64 = ctypes.c_int64


def load(build_if_missing: bool = True):
    """Load libpararnn.so (building it in-tree with nvcc if it is missing or stale)."""
    global _lib
    lib = _lib
    if lib is not None:  # loaded: no lock on the per-call path
        return lib
    with _lock:
        if _lib is None:
            if build_if_missing and _build.needs_build():
                _build.build()
            if not os.path.exists(library_path):
                raise RuntimeError(f"libpararnn.so not found at {library_path}")
            lib = ctypes.CDLL(library_path)
            lib.pararnn_workspace_size.argtypes = [ctypes.c_int, _i64, _i64, _i64, ctypes.c_int32,
                                                   _vp]
            lib.pararnn_workspace_size.restype = ctypes.c_size_t
            for name in ("pararnn_scan_diag", "pararnn_scan_block2"):
                f = getattr(lib, name)
                f.argtypes = [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp, ctypes.c_size_t, _vp, _vp,
                              _vp]
                f.restype = ctypes.c_int
            lib.pararnn_solve_gru.argtypes = [_vp, ctypes.c_int, _vp, _vp, _vp, _i64, _i64, _i64,
                                              ctypes.c_float, ctypes.c_int32, _vp, ctypes.c_size_t,
                                              _vp, _vp, _vp]
            lib.pararnn_solve_gru.restype = ctypes.c_int
            lib.pararnn_solve_lstm.argtypes = [_vp, ctypes.c_int, _vp, _vp, _vp, _vp, _vp, _i64,
                                               _i64, _i64, ctypes.c_float, ctypes.c_int32, _vp,
                                               ctypes.c_size_t, _vp, _vp, _vp]
            lib.pararnn_solve_lstm.restype = ctypes.c_int
            lib.pararnn_solve_gru_backward.argtypes = [_vp, ctypes.c_int, _vp, _vp, _vp, _vp, _vp,
                                                       _vp, _vp, _i64, _i64, _i64, _vp,
                                                       ctypes.c_size_t, _vp, _vp, _vp]
            lib.pararnn_solve_gru_backward.restype = ctypes.c_int
            lib.pararnn_solve_lstm_backward.argtypes = [_vp, ctypes.c_int, _vp, _vp, _vp, _vp, _vp,
                                                        _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64,
                                                        _i64, _vp, ctypes.c_size_t, _vp, _vp, _vp]
            lib.pararnn_solve_lstm_backward.restype = ctypes.c_int
            lib.pararnn_step_gru.argtypes = [_vp, ctypes.c_int, _vp, _vp, _vp, _i64, _i64, _vp]
            lib.pararnn_step_gru.restype = ctypes.c_int
            lib.pararnn_step_lstm.argtypes = [_vp, ctypes.c_int, _vp, _vp, _vp, _vp, _vp, _i64,
                                              _i64, _vp]
            lib.pararnn_step_lstm.restype = ctypes.c_int
            lib.pararnn_rollout_gru.argtypes = [_vp, ctypes.c_int, _vp, _vp, _vp, _i64, _i64, _i64,
                                                _vp]
            lib.pararnn_rollout_gru.restype = ctypes.c_int
            lib.pararnn_rollout_lstm.argtypes = [_vp, ctypes.c_int, _vp, _vp, _vp, _vp, _vp, _i64,
                                                 _i64, _i64, _vp]
            lib.pararnn_rollout_lstm.restype = ctypes.c_int
            lib.pararnn_rollout_mhgru.argtypes = [_vp, ctypes.c_int, _vp, _vp, _vp, _i64, _i64,
                                                  _i64, _vp]
            lib.pararnn_rollout_mhgru.restype = ctypes.c_int
            lib.pararnn_step_mhgru.argtypes = [_vp, ctypes.c_int, _vp, _vp, _vp, _i64, _i64, _vp]
            lib.pararnn_step_mhgru.restype = ctypes.c_int
            lib.pararnn_solve_gru_noalloc.argtypes = [_vp, ctypes.c_int, _vp, _vp, _vp, _i64,
                                                      _i64, _i64, ctypes.c_float, ctypes.c_int32,
                                                      _vp, _vp, _vp]
            lib.pararnn_solve_gru_noalloc.restype = ctypes.c_int
            lib.pararnn_solve_mhgru.argtypes = [_vp, ctypes.c_int, _vp, _vp, _vp, _i64, _i64,
                                                _i64, ctypes.c_float, ctypes.c_int32, _vp,
                                                ctypes.c_size_t, _vp, _vp, _vp]
            lib.pararnn_solve_mhgru.restype = ctypes.c_int
            lib.pararnn_solve_mhgru_strided.argtypes = [_vp, ctypes.c_int, _vp, _vp, _vp, _vp,
                                                        _i64, _i64, _i64, ctypes.c_float,
                                                        ctypes.c_int32, _vp, ctypes.c_size_t,
                                                        _vp, _vp, _vp]
            lib.pararnn_solve_mhgru_strided.restype = ctypes.c_int
            lib.pararnn_input_projection.argtypes = [_vp, _vp, _vp, _vp, ctypes.c_int, _i64,
                                                     _i64, _i64, _vp, _vp]
            lib.pararnn_input_projection.restype = ctypes.c_int
            lib.pararnn_solve_gru_projected.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64,
                                                        _i64, _i64, ctypes.c_float,
                                                        ctypes.c_int32, _vp, ctypes.c_size_t,
                                                        _vp, _vp, _vp]
            lib.pararnn_solve_gru_projected.restype = ctypes.c_int
            lib.pararnn_probe_rate.argtypes = [ctypes.c_int32, ctypes.c_int32, _vp, _vp, _vp]
            lib.pararnn_probe_rate.restype = ctypes.c_int
            _sz, _i32, _f = ctypes.c_size_t, ctypes.c_int32, ctypes.c_float
            lib.pararnn_linattn_workspace_size.argtypes = [_vp, _i32]
            lib.pararnn_linattn_workspace_size.restype = _sz
            lib.pararnn_scan_linattn.argtypes = [_vp] * 10 + [_sz, _vp, _vp, _vp]
            lib.pararnn_scan_linattn.restype = ctypes.c_int
            lib.pararnn_scan_linattn_backward.argtypes = [_vp] * 14 + [_sz, _vp, _vp, _vp]
            lib.pararnn_scan_linattn_backward.restype = ctypes.c_int
            lib.pararnn_step_linattn.argtypes = [_vp] * 4 + [ctypes.c_int] + [_vp] * 5
            lib.pararnn_step_linattn.restype = ctypes.c_int
            lib.pararnn_layer_norm.argtypes = [_vp, ctypes.c_int, _i64, _vp, _vp, _vp,
                                               ctypes.c_int, _vp, _vp, _i64, _i64, _f, _vp]
            lib.pararnn_layer_norm.restype = ctypes.c_int
            lib.pararnn_layer_norm_workspace_size.argtypes = [_i64, _i64]
            lib.pararnn_layer_norm_workspace_size.restype = _sz
            lib.pararnn_layer_norm_backward.argtypes = [_vp, ctypes.c_int, _i64, _vp,
                                                        ctypes.c_int, _i64] + [_vp] * 6 + \
                                                       [_i64, _i64, _vp, _sz, _vp]
            lib.pararnn_layer_norm_backward.restype = ctypes.c_int
            lib.pararnn_status_string.argtypes = [ctypes.c_int]
            lib.pararnn_status_string.restype = ctypes.c_char_p
            lib.pararnn_version.restype = ctypes.c_int32
            _ws_sizes.clear()  # sizes are the loaded library's answers
            _lib = lib
    return _lib


_ws_sizes = {}


def workspace_size(op: int, B: int, L: int, D: int, max_iters: int = 0, opts: Options | None = None):
    """Workspace bytes of a call: the library's answer, remembered per distinct
    argument tuple (options included) until another library is loaded."""
    lib = load()
    key = (int(op), int(B), int(L), int(D), int(max_iters), None if opts is None else bytes(opts))
    n = _ws_sizes.get(key)
    if n is None:
        n = lib.pararnn_workspace_size(int(op), int(B), int(L), int(D), int(max_iters),
                                       ctypes.byref(opts) if opts is not None else None)
        if n == 0:
            raise PararnnError(1, "workspace_size")
        n = int(n)
        if len(_ws_sizes) > 4096:
            _ws_sizes.clear()
        _ws_sizes[key] = n
    return n


def _ptr(t):
    return None if t is None else t.data_ptr()


def _check_dev(name, t, dtype, shape):
    if t is None:
        return
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (no CPU path)")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _one_device(**named):
    """The one CUDA device every given tensor lives on.  The library resolves
    the launch (stream, scratch, occupancy) against the current device, so
    tensors on a device other than the one the call runs on, or on several
    devices, are refused here."""
    dev = None
    first = None
    for name, t in named.items():
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor (no CPU path)")
        if dev is None:
            dev, first = t.device, name
        elif t.device != dev:
            raise ValueError(f"{name} is on {t.device} but {first} is on {dev}: "
                             "all arguments of a call must be on one device")
    if dev is None:
        raise ValueError("no tensor argument")
    return dev


_same_device = contextlib.nullcontext()


def _device_guard(dev):
    """Makes `dev` the current device for the duration of one library call (nothing to
    do where it already is)."""
    if torch.cuda.current_device() == dev.index:
        return _same_device
    return torch.cuda.device(dev)


# the current stream's handle without the object around it (2 us less a call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_handle(stream, dev=None):
    """The stream a call is enqueued on: the given one (which must belong to
    the tensors' device) or that device's current stream."""
    if stream is None:
        if _raw_stream is not None and dev is not None and dev.index is not None:
            return ctypes.c_void_p(_raw_stream(dev.index))
        s = torch.cuda.current_stream(dev)
    else:
        s = stream
        if dev is not None and s.device != dev:
            raise ValueError(f"stream is on {s.device} but the tensors are on {dev}")
    return ctypes.c_void_p(s.cuda_stream)


_ws_cache = threading.local()


def _workspace(nbytes, device, stream=None):
    """Workspace from torch's allocator, reused between calls on the same thread,
    device and stream (calls on one stream run in order, so they can share it;
    calls on different streams get their own)."""
    cache = getattr(_ws_cache, "bufs", None)
    if cache is None:
        cache = _ws_cache.bufs = {}
    dev = device.index if device.index is not None else torch.cuda.current_device()
    s = torch.cuda.current_stream(dev) if stream is None else stream
    key = (dev, s.cuda_stream)
    buf = cache.get(key)
    if buf is None or buf.numel() < nbytes:
        with torch.cuda.stream(s):
            buf = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)
        cache[key] = buf
    return buf


class SolveInfo:
    """Device-side outcome of a solve; fields are read (one device->host copy) on first access."""

    def __init__(self, dev_tensor: torch.Tensor):
        self.tensor = dev_tensor
        self._host = None

    def _get(self):
        if self._host is None:
            raw = self.tensor.cpu().numpy().tobytes()
            self._host = _Info.from_buffer_copy(raw)
        return self._host

    @property
    def iterations(self):
        return int(self._get().iterations)

    @property
    def converged(self):
        return bool(self._get().converged)

    @property
    def status(self):
        return int(self._get().status)

    @property
    def updates(self):
        return int(self._get().updates)

    @property
    def passes(self):
        return int(self._get().passes)

    @property
    def max_residual(self):
        return float(self._get().max_residual)

    @property
    def rho(self):
        h = self._get()
        return [float(h.rho[k]) for k in range(MAX_ITERS + 1)]

    def as_dict(self):
        return dict(iterations=self.iterations, converged=self.converged, status=self.status,
                    updates=self.updates, passes=self.passes, max_residual=self.max_residual)


def _raise(st, where):
    if st != 0:
        raise PararnnError(st, where)


def scan_diag(A, b, h0=None, out=None, status=None, opts: Options | None = None, stream=None):
    """h[b, t, d] = A[b, t, d] * h[b, t-1, d] + b[b, t, d] (fp32, [B, L, D])."""
    lib = load()
    B, L, D = A.shape
    _check_dev("A", A, torch.float32, (B, L, D))
    _check_dev("b", b, torch.float32, (B, L, D))
    _check_dev("h0", h0, torch.float32, (B, D))
    h = torch.empty_like(A) if out is None else out
    _check_dev("out", h, torch.float32, (B, L, D))
    _check_dev("status", status, torch.int32, (1,))
    dev = _one_device(A=A, b=b, h0=h0, out=h, status=status)
    n = workspace_size(OP_SCAN_DIAG, B, L, D, 0, opts)
    ws = _workspace(n, dev, stream)
    with _device_guard(dev):
        st = lib.pararnn_scan_diag(_ptr(A), _ptr(b), _ptr(h0), _ptr(h), B, L, D, _ptr(ws),
                                   ws.numel(), _ptr(status),
                                   ctypes.byref(opts) if opts is not None else None,
                                   _stream_handle(stream, dev))
    _raise(st, "pararnn_scan_diag")
    return h


def scan_block2(A, b, x0=None, out=None, status=None, opts: Options | None = None, stream=None):
    """x_t = A_t x_{t-1} + b_t with A [B, L, D, 2, 2] (row-major) and x, b [B, L, D, 2]."""
    lib = load()
    B, L, D = A.shape[:3]
    _check_dev("A", A, torch.float32, (B, L, D, 2, 2))
    _check_dev("b", b, torch.float32, (B, L, D, 2))
    _check_dev("x0", x0, torch.float32, (B, D, 2))
    x = torch.empty_like(b) if out is None else out
    _check_dev("out", x, torch.float32, (B, L, D, 2))
    _check_dev("status", status, torch.int32, (1,))
    dev = _one_device(A=A, b=b, x0=x0, out=x, status=status)
    n = workspace_size(OP_SCAN_BLOCK2, B, L, D, 0, opts)
    ws = _workspace(n, dev, stream)
    with _device_guard(dev):
        st = lib.pararnn_scan_block2(_ptr(A), _ptr(b), _ptr(x0), _ptr(x), B, L, D, _ptr(ws),
                                     ws.numel(), _ptr(status),
                                     ctypes.byref(opts) if opts is not None else None,
                                     _stream_handle(stream, dev))
    _raise(st, "pararnn_scan_block2")
    return x


def _p_dtype(P):
    if P.dtype == torch.float32:
        return F32
    if P.dtype == torch.bfloat16:
        return BF16
    raise TypeError(f"P must be float32 or bfloat16, got {P.dtype}")


def solve_gru(P, a, h0=None, tol=1e-4, max_iters=32, out=None, info=None,
              opts: Options | None = None, stream=None):
    """ParaGRU Newton solve.  P [B, L, 3, D] (z, r, c), a [3, D] -> (h [B, L, D], SolveInfo)."""
    lib = load()
    B, L, G, D = P.shape
    if G != 3:
        raise ValueError("P must be [B, L, 3, D]")
    dt = _p_dtype(P)
    _check_dev("P", P, P.dtype, (B, L, 3, D))
    _check_dev("a", a, torch.float32, (3, D))
    _check_dev("h0", h0, torch.float32, (B, D))
    h = torch.empty((B, L, D), dtype=torch.float32, device=P.device) if out is None else out
    _check_dev("out", h, torch.float32, (B, L, D))
    if info is None:
        info = torch.empty(INFO_BYTES // 4, dtype=torch.int32, device=P.device)
    _check_dev("info", info, torch.int32, (INFO_BYTES // 4,))
    dev = _one_device(P=P, a=a, h0=h0, out=h, info=info)
    n = workspace_size(OP_GRU, B, L, D, max_iters, opts)
    ws = _workspace(n, dev, stream)
    with _device_guard(dev):
        st = lib.pararnn_solve_gru(_ptr(P), dt, _ptr(a), _ptr(h0), _ptr(h), B, L, D, float(tol),
                                   int(max_iters), _ptr(ws), ws.numel(), _ptr(info),
                                   ctypes.byref(opts) if opts is not None else None,
                                   _stream_handle(stream, dev))
    _raise(st, "pararnn_solve_gru")
    return h, SolveInfo(info)


def solve_mhgru(P, U, h0=None, tol=1e-4, max_iters=32, out=None, info=None,
                opts: Options | None = None, stream=None):
    """Multi-head GRU (dense 8x8 recurrence blocks) Newton solve.  P [B, L, 3, D]
    (z, r, c), U [3, H, 8, 8] with D = 8 H -> (h [B, L, D], SolveInfo)."""
    lib = load()
    B, L, G, D = P.shape
    if G != 3 or U.dim() != 4 or tuple(U.shape[2:]) != (8, 8) or D != 8 * U.shape[1]:
        raise ValueError("P must be [B, L, 3, 8 H] and U [3, H, 8, 8]")
    H = U.shape[1]
    dt = _p_dtype(P)
    _check_dev("P", P, P.dtype, (B, L, 3, D))
    _check_dev("U", U, torch.float32, (3, H, 8, 8))
    _check_dev("h0", h0, torch.float32, (B, D))
    h = torch.empty((B, L, D), dtype=torch.float32, device=P.device) if out is None else out
    _check_dev("out", h, torch.float32, (B, L, D))
    if info is None:
        info = torch.empty(INFO_BYTES // 4, dtype=torch.int32, device=P.device)
    _check_dev("info", info, torch.int32, (INFO_BYTES // 4,))
    dev = _one_device(P=P, U=U, h0=h0, out=h, info=info)
    n = workspace_size(OP_MHGRU, B, L, D, max_iters, opts)
    ws = _workspace(n, dev, stream)
    with _device_guard(dev):
        st = lib.pararnn_solve_mhgru(_ptr(P), dt, _ptr(U), _ptr(h0), _ptr(h), B, L, H,
                                     float(tol), int(max_iters), _ptr(ws), ws.numel(),
                                     _ptr(info), ctypes.byref(opts) if opts is not None else None,
                                     _stream_handle(stream, dev))
    _raise(st, "pararnn_solve_mhgru")
    return h, SolveInfo(info)


def solve_mhgru_strided(P, U, strides, h0=None, tol=1e-4, max_iters=32, out=None, info=None,
                        opts: Options | None = None, stream=None):
    """Multi-head GRU with a time stride per head: head g recurs on h_{t - strides[g]}.
    P [B, L, 3, D] (z, r, c), U [3, H, 8, 8], strides [H] int32 (device, each >= 1)
    -> (h [B, L, D], SolveInfo)."""
    lib = load()
    B, L, G, D = P.shape
    if G != 3 or U.dim() != 4 or tuple(U.shape[2:]) != (8, 8) or D != 8 * U.shape[1]:
        raise ValueError("P must be [B, L, 3, 8 H] and U [3, H, 8, 8]")
    H = U.shape[1]
    dt = _p_dtype(P)
    _check_dev("P", P, P.dtype, (B, L, 3, D))
    _check_dev("U", U, torch.float32, (3, H, 8, 8))
    _check_dev("strides", strides, torch.int32, (H,))
    _check_dev("h0", h0, torch.float32, (B, D))
    h = torch.empty((B, L, D), dtype=torch.float32, device=P.device) if out is None else out
    _check_dev("out", h, torch.float32, (B, L, D))
    if info is None:
        info = torch.empty(INFO_BYTES // 4, dtype=torch.int32, device=P.device)
    _check_dev("info", info, torch.int32, (INFO_BYTES // 4,))
    dev = _one_device(P=P, U=U, strides=strides, h0=h0, out=h, info=info)
    n = workspace_size(OP_MHGRU_STRIDED, B, L, D, max_iters, opts)
    ws = _workspace(n, dev, stream)
    with _device_guard(dev):
        st = lib.pararnn_solve_mhgru_strided(_ptr(P), dt, _ptr(U), _ptr(strides), _ptr(h0),
                                             _ptr(h), B, L, H, float(tol), int(max_iters),
                                             _ptr(ws), ws.numel(), _ptr(info),
                                             ctypes.byref(opts) if opts is not None else None,
                                             _stream_handle(stream, dev))
    _raise(st, "pararnn_solve_mhgru_strided")
    return h, SolveInfo(info)


def solve_lstm(P, a, c0=None, h0=None, tol=1e-4, max_iters=32, out=None, info=None,
               opts: Options | None = None, stream=None):
    """ParaLSTM Newton solve.  P [B, L, 4, D] (i, f, g, o), a [4, D] -> (c, h, SolveInfo)."""
    lib = load()
    B, L, G, D = P.shape
    if G != 4:
        raise ValueError("P must be [B, L, 4, D]")
    dt = _p_dtype(P)
    _check_dev("P", P, P.dtype, (B, L, 4, D))
    _check_dev("a", a, torch.float32, (4, D))
    _check_dev("c0", c0, torch.float32, (B, D))
    _check_dev("h0", h0, torch.float32, (B, D))
    if out is None:
        c = torch.empty((B, L, D), dtype=torch.float32, device=P.device)
        h = torch.empty((B, L, D), dtype=torch.float32, device=P.device)
    else:
        c, h = out
    _check_dev("c", c, torch.float32, (B, L, D))
    _check_dev("h", h, torch.float32, (B, L, D))
    if info is None:
        info = torch.empty(INFO_BYTES // 4, dtype=torch.int32, device=P.device)
    _check_dev("info", info, torch.int32, (INFO_BYTES // 4,))
    dev = _one_device(P=P, a=a, c0=c0, h0=h0, c=c, h=h, info=info)
    n = workspace_size(OP_LSTM, B, L, D, max_iters, opts)
    ws = _workspace(n, dev, stream)
    with _device_guard(dev):
        st = lib.pararnn_solve_lstm(_ptr(P), dt, _ptr(a), _ptr(c0), _ptr(h0), _ptr(c), _ptr(h),
                                    B, L, D, float(tol), int(max_iters), _ptr(ws), ws.numel(),
                                    _ptr(info), ctypes.byref(opts) if opts is not None else None,
                                    _stream_handle(stream, dev))
    _raise(st, "pararnn_solve_lstm")
    return c, h, SolveInfo(info)


def solve_gru_projected(x, W, bias, a, h0=None, tol=1e-4, max_iters=32, out=None, info=None,
                        opts: Options | None = None, stream=None):
    """ParaGRU layer from its inputs: P = x W^T + bias on the tensor cores, fused
    with the Newton solve so that P never reaches HBM.  x [B, L, K] bf16, W
    [3 D, K] bf16 (rows z, r, c), bias [3 D] fp32 or None, a [3, D] ->
    (h [B, L, D], SolveInfo)."""
    lib = load()
    if x.dim() != 3 or W.dim() != 2 or x.shape[-1] != W.shape[1] or W.shape[0] % 3 != 0:
        raise ValueError(f"x [B, L, K] and W [3 D, K] do not match: {tuple(x.shape)}, "
                         f"{tuple(W.shape)}")
    B, L, K = x.shape
    D = W.shape[0] // 3
    _check_dev("x", x, torch.bfloat16, (B, L, K))
    _check_dev("W", W, torch.bfloat16, (3 * D, K))
    _check_dev("bias", bias, torch.float32, (3 * D,))
    _check_dev("a", a, torch.float32, (3, D))
    _check_dev("h0", h0, torch.float32, (B, D))
    h = torch.empty((B, L, D), dtype=torch.float32, device=x.device) if out is None else out
    _check_dev("out", h, torch.float32, (B, L, D))
    if info is None:
        info = torch.empty(INFO_BYTES // 4, dtype=torch.int32, device=x.device)
    _check_dev("info", info, torch.int32, (INFO_BYTES // 4,))
    dev = _one_device(x=x, W=W, bias=bias, a=a, h0=h0, out=h, info=info)
    n = workspace_size(OP_GRU_PROJECTED, B, L, D, max_iters, opts)
    ws = _workspace(n, dev, stream)
    with _device_guard(dev):
        st = lib.pararnn_solve_gru_projected(_ptr(x), _ptr(W), _ptr(bias), _ptr(a), _ptr(h0),
                                             _ptr(h), B, L, D, K, float(tol), int(max_iters),
                                             _ptr(ws), ws.numel(), _ptr(info),
                                             ctypes.byref(opts) if opts is not None else None,
                                             _stream_handle(stream, dev))
    _raise(st, "pararnn_solve_gru_projected")
    return h, SolveInfo(info)


NOALLOC_SCRATCH_BYTES = 4 << 20


def solve_gru_noalloc(P, a, h0=None, tol=1e-4, max_iters=32, out=None, info=None,
                      opts: Options | None = None, stream=None):
    """ParaGRU Newton solve through ``pararnn_solve_gru_noalloc``: the library
    allocates nothing and uses its own fixed device scratch array instead of a
    workspace (for callers that cannot allocate device memory where they
    solve).  Calls on one device share that array, so they must not overlap on
    the GPU.  ``out`` and ``info`` may be passed to keep this call itself free
    of allocations."""
    lib = load()
    B, L, G, D = P.shape
    if G != 3:
        raise ValueError("P must be [B, L, 3, D]")
    dt = _p_dtype(P)
    _check_dev("P", P, P.dtype, (B, L, 3, D))
    _check_dev("a", a, torch.float32, (3, D))
    _check_dev("h0", h0, torch.float32, (B, D))
    h = torch.empty((B, L, D), dtype=torch.float32, device=P.device) if out is None else out
    _check_dev("out", h, torch.float32, (B, L, D))
    if info is None:
        info = torch.empty(INFO_BYTES // 4, dtype=torch.int32, device=P.device)
    _check_dev("info", info, torch.int32, (INFO_BYTES // 4,))
    dev = _one_device(P=P, a=a, h0=h0, out=h, info=info)
    with _device_guard(dev):
        st = lib.pararnn_solve_gru_noalloc(_ptr(P), dt, _ptr(a), _ptr(h0), _ptr(h), B, L, D,
                                           float(tol), int(max_iters), _ptr(info),
                                           ctypes.byref(opts) if opts is not None else None,
                                           _stream_handle(stream, dev))
    _raise(st, "pararnn_solve_gru_noalloc")
    return h, SolveInfo(info)


def solve_gru_backward(P, a, h, dh, h0=None, out=None, status=None,
                       opts: Options | None = None, stream=None):
    """Gradients of a loss through the ParaGRU solution h, given dh = dl/dh.

    Returns (dP [B, L, 3, D] fp32, da [3, D], dh0 [B, D])."""
    lib = load()
    B, L, G, D = P.shape
    if G != 3:
        raise ValueError("P must be [B, L, 3, D]")
    dt = _p_dtype(P)
    _check_dev("P", P, P.dtype, (B, L, 3, D))
    _check_dev("a", a, torch.float32, (3, D))
    _check_dev("h0", h0, torch.float32, (B, D))
    _check_dev("h", h, torch.float32, (B, L, D))
    _check_dev("dh", dh, torch.float32, (B, L, D))
    if out is None:
        dP = torch.empty((B, L, 3, D), dtype=torch.float32, device=P.device)
        da = torch.empty((3, D), dtype=torch.float32, device=P.device)
        dh0 = torch.empty((B, D), dtype=torch.float32, device=P.device)
    else:
        dP, da, dh0 = out
    _check_dev("dP", dP, torch.float32, (B, L, 3, D))
    _check_dev("da", da, torch.float32, (3, D))
    _check_dev("dh0", dh0, torch.float32, (B, D))
    _check_dev("status", status, torch.int32, (1,))
    dev = _one_device(P=P, a=a, h0=h0, h=h, dh=dh, dP=dP, da=da, dh0=dh0, status=status)
    n = workspace_size(OP_GRU_BACKWARD, B, L, D, 0, opts)
    ws = _workspace(n, dev, stream)
    with _device_guard(dev):
        st = lib.pararnn_solve_gru_backward(_ptr(P), dt, _ptr(a), _ptr(h0), _ptr(h), _ptr(dh),
                                            _ptr(dP), _ptr(da), _ptr(dh0), B, L, D, _ptr(ws),
                                            ws.numel(), _ptr(status),
                                            ctypes.byref(opts) if opts is not None else None,
                                            _stream_handle(stream, dev))
    _raise(st, "pararnn_solve_gru_backward")
    return dP, da, dh0


def solve_lstm_backward(P, a, c, h, dc, dh, c0=None, h0=None, out=None, status=None,
                        opts: Options | None = None, stream=None):
    """Gradients through the ParaLSTM solution (c, h), given dc = dl/dc and dh = dl/dh
    (either may be None).  Returns (dP [B, L, 4, D], da [4, D], dc0 [B, D], dh0 [B, D])."""
    lib = load()
    B, L, G, D = P.shape
    if G != 4:
        raise ValueError("P must be [B, L, 4, D]")
    dt = _p_dtype(P)
    _check_dev("P", P, P.dtype, (B, L, 4, D))
    _check_dev("a", a, torch.float32, (4, D))
    for nm, t in (("c0", c0), ("h0", h0)):
        _check_dev(nm, t, torch.float32, (B, D))
    for nm, t in (("c", c), ("h", h), ("dc", dc), ("dh", dh)):
        _check_dev(nm, t, torch.float32, (B, L, D))
    if out is None:
        dP = torch.empty((B, L, 4, D), dtype=torch.float32, device=P.device)
        da = torch.empty((4, D), dtype=torch.float32, device=P.device)
        dc0 = torch.empty((B, D), dtype=torch.float32, device=P.device)
        dh0 = torch.empty((B, D), dtype=torch.float32, device=P.device)
    else:
        dP, da, dc0, dh0 = out
    _check_dev("dP", dP, torch.float32, (B, L, 4, D))
    _check_dev("da", da, torch.float32, (4, D))
    _check_dev("dc0", dc0, torch.float32, (B, D))
    _check_dev("dh0", dh0, torch.float32, (B, D))
    _check_dev("status", status, torch.int32, (1,))
    dev = _one_device(P=P, a=a, c0=c0, h0=h0, c=c, h=h, dc=dc, dh=dh, dP=dP, da=da, dc0=dc0,
                      dh0=dh0, status=status)
    n = workspace_size(OP_LSTM_BACKWARD, B, L, D, 0, opts)
    ws = _workspace(n, dev, stream)
    with _device_guard(dev):
        st = lib.pararnn_solve_lstm_backward(_ptr(P), dt, _ptr(a), _ptr(c0), _ptr(h0), _ptr(c),
                                             _ptr(h), _ptr(dc), _ptr(dh), _ptr(dP), _ptr(da),
                                             _ptr(dc0), _ptr(dh0), B, L, D, _ptr(ws), ws.numel(),
                                             _ptr(status),
                                             ctypes.byref(opts) if opts is not None else None,
                                             _stream_handle(stream, dev))
    _raise(st, "pararnn_solve_lstm_backward")
    return dP, da, dc0, dh0


def step_gru(P, a, h_prev=None, out=None, stream=None):
    """One ParaGRU step for every channel (decode): P [B, 3, D] -> h_next [B, D]."""
    lib = load()
    B, G, D = P.shape
    if G != 3:
        raise ValueError("P must be [B, 3, D]")
    dt = _p_dtype(P)
    _check_dev("P", P, P.dtype, (B, 3, D))
    _check_dev("a", a, torch.float32, (3, D))
    _check_dev("h_prev", h_prev, torch.float32, (B, D))
    h = torch.empty((B, D), dtype=torch.float32, device=P.device) if out is None else out
    _check_dev("out", h, torch.float32, (B, D))
    dev = _one_device(P=P, a=a, h_prev=h_prev, out=h)
    with _device_guard(dev):
        st = lib.pararnn_step_gru(_ptr(P), dt, _ptr(a), _ptr(h_prev), _ptr(h), B, D,
                                  _stream_handle(stream, dev))
    _raise(st, "pararnn_step_gru")
    return h


def step_mhgru(P, U, h_prev=None, out=None, stream=None):
    """One multi-head GRU step (decode): P [B, 3, D] (z, r, c), U [3, H, 8, 8],
    D = 8 H -> h_next [B, D]."""
    lib = load()
    B, G, D = P.shape
    if G != 3 or U.dim() != 4 or tuple(U.shape[2:]) != (8, 8) or D != 8 * U.shape[1]:
        raise ValueError("P must be [B, 3, 8 H] and U [3, H, 8, 8]")
    H = U.shape[1]
    dt = _p_dtype(P)
    _check_dev("P", P, P.dtype, (B, 3, D))
    _check_dev("U", U, torch.float32, (3, H, 8, 8))
    _check_dev("h_prev", h_prev, torch.float32, (B, D))
    h = torch.empty((B, D), dtype=torch.float32, device=P.device) if out is None else out
    _check_dev("out", h, torch.float32, (B, D))
    dev = _one_device(P=P, U=U, h_prev=h_prev, out=h)
    with _device_guard(dev):
        st = lib.pararnn_step_mhgru(_ptr(P), dt, _ptr(U), _ptr(h_prev), _ptr(h), B, H,
                                    _stream_handle(stream, dev))
    _raise(st, "pararnn_step_mhgru")
    return h


def input_projection(x, W, bias=None, out=None, out_dtype=torch.float32, status=None,
                     stream=None):
    """P = x W^T + bias on the tensor cores: x [..., K] bf16, W [N, K] bf16,
    bias [N] fp32 or None -> P [..., N] (fp32 or bf16).  With N = G * D and x
    [B, L, K], P.view(B, L, G, D) is the solve's input."""
    lib = load()
    if x.dtype != torch.bfloat16 or W.dtype != torch.bfloat16:
        raise TypeError("x and W must be bf16")
    if W.dim() != 2 or x.shape[-1] != W.shape[1]:
        raise ValueError(f"x [..., K] and W [N, K] do not match: {tuple(x.shape)}, {tuple(W.shape)}")
    if out_dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("out_dtype must be float32 or bfloat16")
    N, K = W.shape
    lead = tuple(x.shape[:-1])
    M = 1
    for n in lead:
        M *= n
    if not x.is_contiguous() or not W.is_contiguous():
        raise ValueError("x and W must be contiguous")
    _check_dev("x", x, torch.bfloat16, lead + (K,))
    _check_dev("W", W, torch.bfloat16, (N, K))
    _check_dev("bias", bias, torch.float32, (N,))
    P = torch.empty(lead + (N,), dtype=out_dtype, device=x.device) if out is None else out
    _check_dev("out", P, out_dtype, lead + (N,))
    _check_dev("status", status, torch.int32, (1,))
    dt = BF16 if out_dtype == torch.bfloat16 else F32
    dev = _one_device(x=x, W=W, bias=bias, out=P, status=status)
    with _device_guard(dev):
        st = lib.pararnn_input_projection(_ptr(x), _ptr(W), _ptr(bias), _ptr(P), dt, M, N, K,
                                          _ptr(status), _stream_handle(stream, dev))
    _raise(st, "pararnn_input_projection")
    return P


def step_lstm(P, a, c_prev=None, h_prev=None, out=None, stream=None):
    """One ParaLSTM step for every channel: P [B, 4, D] -> (c_next, h_next)."""
    lib = load()
    B, G, D = P.shape
    if G != 4:
        raise ValueError("P must be [B, 4, D]")
    dt = _p_dtype(P)
    _check_dev("P", P, P.dtype, (B, 4, D))
    _check_dev("a", a, torch.float32, (4, D))
    _check_dev("c_prev", c_prev, torch.float32, (B, D))
    _check_dev("h_prev", h_prev, torch.float32, (B, D))
    if out is None:
        c = torch.empty((B, D), dtype=torch.float32, device=P.device)
        h = torch.empty((B, D), dtype=torch.float32, device=P.device)
    else:
        c, h = out
    _check_dev("c", c, torch.float32, (B, D))
    _check_dev("h", h, torch.float32, (B, D))
    dev = _one_device(P=P, a=a, c_prev=c_prev, h_prev=h_prev, c=c, h=h)
    with _device_guard(dev):
        st = lib.pararnn_step_lstm(_ptr(P), dt, _ptr(a), _ptr(c_prev), _ptr(h_prev), _ptr(c),
                                   _ptr(h), B, D, _stream_handle(stream, dev))
    _raise(st, "pararnn_step_lstm")
    return c, h


def rollout_gru(P, a, h0=None, out=None, stream=None):
    """Sequential ParaGRU application on the GPU (one thread per channel)."""
    lib = load()
    B, L, G, D = P.shape
    if G != 3:
        raise ValueError("P must be [B, L, 3, D]")
    dt = _p_dtype(P)
    _check_dev("P", P, P.dtype, (B, L, 3, D))
    _check_dev("a", a, torch.float32, (3, D))
    _check_dev("h0", h0, torch.float32, (B, D))
    h = torch.empty((B, L, D), dtype=torch.float32, device=P.device) if out is None else out
    _check_dev("out", h, torch.float32, (B, L, D))
    dev = _one_device(P=P, a=a, h0=h0, out=h)
    with _device_guard(dev):
        st = lib.pararnn_rollout_gru(_ptr(P), dt, _ptr(a), _ptr(h0), _ptr(h), B, L, D,
                                     _stream_handle(stream, dev))
    _raise(st, "pararnn_rollout_gru")
    return h


def rollout_mhgru(P, U, h0=None, out=None, stream=None):
    """Sequential multi-head GRU application on the GPU (8 lanes per head
    sequence).  P [B, L, 3, D] (z, r, c), U [3, H, 8, 8], D = 8 H -> h [B, L, D]."""
    lib = load()
    B, L, G, D = P.shape
    if G != 3 or U.dim() != 4 or tuple(U.shape[2:]) != (8, 8) or D != 8 * U.shape[1]:
        raise ValueError("P must be [B, L, 3, 8 H] and U [3, H, 8, 8]")
    H = U.shape[1]
    dt = _p_dtype(P)
    _check_dev("P", P, P.dtype, (B, L, 3, D))
    _check_dev("U", U, torch.float32, (3, H, 8, 8))
    _check_dev("h0", h0, torch.float32, (B, D))
    h = torch.empty((B, L, D), dtype=torch.float32, device=P.device) if out is None else out
    _check_dev("out", h, torch.float32, (B, L, D))
    dev = _one_device(P=P, U=U, h0=h0, out=h)
    with _device_guard(dev):
        st = lib.pararnn_rollout_mhgru(_ptr(P), dt, _ptr(U), _ptr(h0), _ptr(h), B, L, H,
                                       _stream_handle(stream, dev))
    _raise(st, "pararnn_rollout_mhgru")
    return h


def rollout_lstm(P, a, c0=None, h0=None, out=None, stream=None):
    """Sequential ParaLSTM application on the GPU (one thread per channel)."""
    lib = load()
    B, L, G, D = P.shape
    if G != 4:
        raise ValueError("P must be [B, L, 4, D]")
    dt = _p_dtype(P)
    _check_dev("P", P, P.dtype, (B, L, 4, D))
    _check_dev("a", a, torch.float32, (4, D))
    _check_dev("c0", c0, torch.float32, (B, D))
    _check_dev("h0", h0, torch.float32, (B, D))
    if out is None:
        c = torch.empty((B, L, D), dtype=torch.float32, device=P.device)
        h = torch.empty((B, L, D), dtype=torch.float32, device=P.device)
    else:
        c, h = out
    _check_dev("c", c, torch.float32, (B, L, D))
    _check_dev("h", h, torch.float32, (B, L, D))
    dev = _one_device(P=P, a=a, c0=c0, h0=h0, c=c, h=h)
    with _device_guard(dev):
        st = lib.pararnn_rollout_lstm(_ptr(P), dt, _ptr(a), _ptr(c0), _ptr(h0), _ptr(c), _ptr(h),
                                      B, L, D, _stream_handle(stream, dev))
    _raise(st, "pararnn_rollout_lstm")
    return c, h


def _stream_strides(name, t, dtype, shape, unit):
    """Checks one stream of a linear-attention call and returns its element
    strides.  The last axis is contiguous; with ``unit`` > 1 every stride is a
    positive multiple of it (what the tensor copies need).  An axis of size 1
    takes the stride of a dense layout."""
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    sizes, strides = t.shape, list(t.stride())
    if sizes != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(sizes)}")
    if strides[-1] != 1 and t.numel() > 0:
        raise ValueError(f"{name}: the last axis must be contiguous")
    dense = sizes[-1]
    for i in range(len(strides) - 2, -1, -1):
        n = sizes[i]
        if n <= 1:
            strides[i] = dense
        elif unit > 1 and (strides[i] <= 0 or strides[i] % unit) and t.numel() > 0:
            raise ValueError(f"{name}: strides must be positive multiples of {unit} elements, "
                             f"got {tuple(t.stride())}")
        else:
            dense *= n
    strides = strides[:-1]
    if len(strides) == 2:  # one token: its stride is not used
        strides.insert(1, 0)
    return _Stride3(*strides)


_linattn_descs = {}


def _linattn_desc(q, k, v, log_decay, scale, dtype, do=None):
    """The call's descriptor from its tensors ([B, L, heads, size], or [B, heads,
    size] for one token), remembered per shapes, strides and types.  Scans need
    strides and first elements on 16-byte units.  Its ``bytes`` are the extents of q, k
    and v."""
    tokens = q.dim() == 4
    key = (q.shape, k.shape, v.shape, log_decay.shape, q.stride(), k.stride(), v.stride(),
           log_decay.stride(), q.dtype, k.dtype, v.dtype, log_decay.dtype, dtype, scale,
           None if do is None else (do.shape, do.stride(), do.dtype))
    d = _linattn_descs.get(key)
    if d is None:
        if q.dim() not in (3, 4) or k.dim() != q.dim() or v.dim() != q.dim() \
                or log_decay.dim() != 1:
            raise ValueError("q, k, v must be [B, L, heads, size] ([B, heads, size] for one "
                             "token) and log_decay [H]")
        lead, unit = tuple(q.shape[:-2]), 8 if tokens else 1
        Hq, Dk = q.shape[-2:]
        Hk, (Hv, Dv), H = k.shape[-2], v.shape[-2:], log_decay.shape[0]
        if H == 0 or min(Hq, Hk, Hv) == 0 or H % Hq or H % Hk or H % Hv:
            raise ValueError(f"the heads of q, k and v ({Hq}, {Hk}, {Hv}) must divide the {H} "
                             "heads of log_decay")
        if Dk % 8 or Dv % 8 or not 8 <= Dk <= 128 or not 8 <= Dv <= 128:
            raise ValueError(f"head sizes must be multiples of 8 from 8 to 128, got {Dk} and {Dv}")
        if log_decay.dtype != torch.float32:
            raise TypeError(f"log_decay: expected {torch.float32}, got {log_decay.dtype}")
        if not log_decay.is_contiguous():
            raise ValueError("log_decay must be contiguous")
        d = _LinAttn(lead[0], lead[1] if tokens else 1, H, Hq, Hk, Hv, Dk, Dv, scale, 0,
                     _stream_strides("q", q, dtype, lead + (Hq, Dk), unit),
                     _stream_strides("k", k, dtype, lead + (Hk, Dk), unit),
                     _stream_strides("v", v, dtype, lead + (Hv, Dv), unit))
        d.bytes = tuple(hi - lo for lo, hi in map(_extent, (q, k, v)))
        if do is not None:
            d.do_stride = _stream_strides("do", do, dtype, lead + (H, Dv), unit)
        if len(_linattn_descs) > 1024:
            _linattn_descs.clear()
        _linattn_descs[key] = d
    if tokens:
        for name, t in (("q", q), ("k", k), ("v", v), ("do", do)):
            if t is not None and t.data_ptr() % 16:
                raise ValueError(f"{name} must start on a 16-byte boundary")
    return d


def _linattn_ws(lib, d, backward):
    """Workspace bytes of a scan with this descriptor: the library's answer, remembered
    like those of the solves."""
    key = ("linattn", d.B, d.L, d.H, d.Hq, d.Hk, d.Hv, d.Dk, d.Dv, backward)
    n = _ws_sizes.get(key)
    if n is None:
        n = int(lib.pararnn_linattn_workspace_size(ctypes.byref(d), backward))
        if len(_ws_sizes) > 4096:
            _ws_sizes.clear()
        _ws_sizes[key] = n
    return n


def _making_on(stream):
    """Where a call's own outputs are made: on the stream that it runs on."""
    return _same_device if stream is None else torch.cuda.stream(stream)


def _call_buffer(nbytes, device, stream):
    """Workspace of one call, from torch's allocator for the stream it runs on (None
    where the call needs none: the library then says 256).  Taken anew each call,
    so that captured graphs keep workspaces of their own."""
    if nbytes <= 256:
        return None
    with _making_on(stream):
        return torch.empty(nbytes, dtype=torch.uint8, device=device)


def _extent(t):
    """First byte of a tensor and the one behind its last (strides are not negative)."""
    p = t.data_ptr()
    if t.is_contiguous():
        return p, p + t.nbytes
    if t.numel() == 0:
        return p, p
    last = sum((n - 1) * st for n, st in zip(t.shape, t.stride()))
    return p, p + (last + 1) * t.element_size()


def _apart(outputs, inputs, same=()):
    """Refuses outputs of the caller's that lie over each other or over an input, but for
    the pairs of names in ``same``, which may be one and the same tensor."""
    seen = [(n, *_extent(t)) for n, t in inputs if t is not None]
    for name, t in outputs:
        if t is None:
            continue
        lo, hi = _extent(t)
        for other, lo2, hi2 in seen:
            if lo < hi2 and lo2 < hi:
                alias = (name, other) in same
                if not (alias and lo == lo2):
                    raise ValueError(f"{name} must " + (f"be {other} itself or " if alias else "")
                                     + f"not overlap {other}")
        seen.append((name, lo, hi))


def _linattn_apart(d, q, k, v, log_decay, state, out, state_out, name, lengths=None, status=None):
    """``_apart`` for a forward call, by numbers first: it stands before every decode step."""
    po, ps, pi = out.data_ptr(), state_out.data_ptr(), 0 if state is None else state.data_ptr()
    rows, item = d.B * d.H * d.Dv, out.element_size()
    eo, es = po + rows * d.L * item, ps + rows * d.Dk * 4
    bq, bk, bv = d.bytes
    apart = not (po < es and ps < eo) and (pi in (0, ps) or not (ps < pi + es - ps and pi < es)) \
        and (pi == 0 or not (po < pi + es - ps and pi < eo))
    reads = [(q.data_ptr(), bq), (k.data_ptr(), bk), (v.data_ptr(), bv),
             (log_decay.data_ptr(), 4 * d.H)]
    if lengths is not None:
        reads.append((lengths.data_ptr(), 4 * d.B))
    if status is not None:  # written besides: apart from what is read, too
        reads.append((status.data_ptr(), 4))
        apart = apart and all(status.data_ptr() + 4 <= u or u + n <= status.data_ptr()
                              for u, n in reads[:-1] + [(pi, es - ps if pi else 0)])
    for u, n in reads:
        apart = apart and not (po < u + n and u < eo or ps < u + n and u < es)
    if not apart:
        _apart((("out", out), ("state_out", state_out), ("status", status)),
               (("q", q), ("k", k), ("v", v), ("log_decay", log_decay), (name, state),
                ("lengths", lengths)),
               same=(("state_out", name),))


def scan_linattn(q, k, v, log_decay, s0=None, scale=1.0, lengths=None, out=None, state_out=None,
                 status=None, opts: Options | None = None, stream=None):
    """Linear attention with one decay per head over a prompt:
    S_t = exp(log_decay) S_{t-1} + k_t^T v_t, o_t = scale q_t S_t.

    q [B, L, Hq, Dk], k [B, L, Hk, Dk], v [B, L, Hv, Dv] bf16 (strided views allowed,
    last axis contiguous), log_decay [H] fp32, s0 [B, H, Dk, Dv] fp32 or None ->
    (o [B, L, H, Dv] bf16, s [B, H, Dk, Dv] fp32).  lengths [B] int32 (device): tokens
    at and after a row's length are not used; their rows of o are left as they were
    in ``out`` and are zero in a tensor this call makes.  ``state_out`` may be s0; outputs
    lie over no other argument.  ``status`` [1] int32 (device) is 0, or 4 where a wait on the
    device ran out (``opts.wait_timeout_ns``): the results are then undefined.  Nothing is
    raised for that, the call does not wait for the device."""
    lib = load()
    if q.dim() != 4:
        raise ValueError("q, k, v must be [B, L, heads, size]")
    d = _linattn_desc(q, k, v, log_decay, float(scale), torch.bfloat16)
    B, L, H, Dk, Dv = d.B, d.L, d.H, d.Dk, d.Dv
    _check_dev("s0", s0, torch.float32, (B, H, Dk, Dv))
    _check_dev("lengths", lengths, torch.int32, (B,))
    _check_dev("out", out, torch.bfloat16, (B, L, H, Dv))
    _check_dev("state_out", state_out, torch.float32, (B, H, Dk, Dv))
    _check_dev("status", status, torch.int32, (1,))
    dev = _one_device(q=q, k=k, v=v, log_decay=log_decay, s0=s0, lengths=lengths, out=out,
                      state_out=state_out, status=status)
    given = out is not None or state_out is not None
    with _making_on(stream):
        if out is None:
            out = (q.new_empty if lengths is None else q.new_zeros)((B, L, H, Dv))
        if state_out is None:
            state_out = log_decay.new_empty((B, H, Dk, Dv))
    if given or status is not None:
        _linattn_apart(d, q, k, v, log_decay, s0, out, state_out, "s0", lengths, status)
    nws = _linattn_ws(lib, d, 0)
    ws = _call_buffer(nws, dev, stream)
    with _device_guard(dev):
        st = lib.pararnn_scan_linattn(ctypes.byref(d), _ptr(q), _ptr(k), _ptr(v), _ptr(log_decay),
                                      _ptr(s0), _ptr(lengths), _ptr(out), _ptr(state_out),
                                      _ptr(ws), nws, _ptr(status),
                                      ctypes.byref(opts) if opts is not None else None,
                                      _stream_handle(stream, dev))
    _raise(st, "pararnn_scan_linattn")
    return out, state_out


def scan_linattn_backward(q, k, v, log_decay, do, s0=None, ds=None, scale=1.0, lengths=None,
                          out=None, status=None, opts: Options | None = None, stream=None):
    """Gradients of a loss through ``scan_linattn``, given do = dl/do [B, L, H, Dv] bf16
    and ds = dl/ds of the final state (or None): (dq, dk, dv bf16 in the shapes of q, k
    and v, summed over the heads that share one; ds0 [B, H, Dk, Dv] fp32).  Rows at and
    after a batch row's length get zeros.  The decay is a constant of the layer.  Outputs lie
    over no other argument; ``status`` as in ``scan_linattn``."""
    lib = load()
    if q.dim() != 4 or do.dim() != 4:
        raise ValueError("q, k, v and do must be [B, L, heads, size]")
    d = _linattn_desc(q, k, v, log_decay, float(scale), torch.bfloat16, do)
    B, L, H, Dk, Dv = d.B, d.L, d.H, d.Dk, d.Dv
    _check_dev("s0", s0, torch.float32, (B, H, Dk, Dv))
    _check_dev("ds", ds, torch.float32, (B, H, Dk, Dv))
    _check_dev("lengths", lengths, torch.int32, (B,))
    _check_dev("status", status, torch.int32, (1,))
    dev = _one_device(q=q, k=k, v=v, log_decay=log_decay, do=do, s0=s0, ds=ds, lengths=lengths,
                      status=status)
    outputs = () if status is None else (("status", status),)
    if out is None:
        with _making_on(stream):
            dq, dk, dv = q.new_empty(q.shape), q.new_empty(k.shape), q.new_empty(v.shape)
            ds0 = log_decay.new_empty((B, H, Dk, Dv))
    else:
        dq, dk, dv, ds0 = out
        for name, t, like in (("dq", dq, q), ("dk", dk, k), ("dv", dv, v)):
            _check_dev(name, t, torch.bfloat16, like.shape)
        _check_dev("ds0", ds0, torch.float32, (B, H, Dk, Dv))
        _one_device(q=q, dq=dq, dk=dk, dv=dv, ds0=ds0)
        outputs += (("dq", dq), ("dk", dk), ("dv", dv), ("ds0", ds0))
    if outputs:
        _apart(outputs, (("q", q), ("k", k), ("v", v), ("log_decay", log_decay), ("do", do),
                         ("s0", s0), ("ds", ds), ("lengths", lengths)))
    nws = _linattn_ws(lib, d, 1)
    ws = _call_buffer(nws, dev, stream)
    with _device_guard(dev):
        st = lib.pararnn_scan_linattn_backward(
            ctypes.byref(d), _ptr(q), _ptr(k), _ptr(v), _ptr(log_decay), _ptr(s0), _ptr(do),
            _ptr(ds), _ptr(lengths), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(ds0), _ptr(ws),
            nws, _ptr(status), ctypes.byref(opts) if opts is not None else None,
            _stream_handle(stream, dev))
    _raise(st, "pararnn_scan_linattn_backward")
    return dq, dk, dv, ds0


def step_linattn(q, k, v, log_decay, s_prev=None, scale=1.0, out=None, state_out=None,
                 stream=None):
    """One token of linear attention (decode): s = exp(log_decay) s_prev + k^T v,
    o = scale q s.  q [B, Hq, Dk], k [B, Hk, Dk], v [B, Hv, Dv] all fp32 or all bf16
    (last axis contiguous), s_prev [B, H, Dk, Dv] fp32 or None -> (o [B, H, Dv] of
    their type, s).  ``state_out`` may be s_prev: the state is then updated in place."""
    lib = load()
    dt = F32 if q.dtype == torch.float32 else BF16
    if q.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"q must be float32 or bfloat16, got {q.dtype}")
    if q.dim() != 3:
        raise ValueError("q, k, v must be [B, heads, size]")
    d = _linattn_desc(q, k, v, log_decay, float(scale), q.dtype)
    B, H, Dk, Dv = d.B, d.H, d.Dk, d.Dv
    _check_dev("s_prev", s_prev, torch.float32, (B, H, Dk, Dv))
    _check_dev("out", out, q.dtype, (B, H, Dv))
    _check_dev("state_out", state_out, torch.float32, (B, H, Dk, Dv))
    dev = _one_device(q=q, k=k, v=v, log_decay=log_decay, s_prev=s_prev, out=out,
                      state_out=state_out)
    given = out is not None or state_out is not None
    with _making_on(stream):
        if out is None:
            out = q.new_empty((B, H, Dv))
        if state_out is None:
            state_out = log_decay.new_empty((B, H, Dk, Dv))
    if given:
        _linattn_apart(d, q, k, v, log_decay, s_prev, out, state_out, "s_prev")
    with _device_guard(dev):
        st = lib.pararnn_step_linattn(ctypes.byref(d), _ptr(q), _ptr(k), _ptr(v), dt,
                                      _ptr(log_decay), _ptr(s_prev), _ptr(out), _ptr(state_out),
                                      _stream_handle(stream, dev))
    _raise(st, "pararnn_step_linattn")
    return out, state_out


def _norm_dtype(name, t):
    if t.dtype == torch.float32:
        return F32
    if t.dtype == torch.bfloat16:
        return BF16
    raise TypeError(f"{name} must be float32 or bfloat16, got {t.dtype}")


def _rows(name, t):
    """(rows, row stride) of a tensor whose last axis is contiguous and whose
    leading axes are evenly spaced rows."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (no CPU path)")
    if t.dim() == 0 or t.shape[-1] == 0:
        raise ValueError(f"{name} must have a last axis of at least one element")
    if t.is_contiguous():
        return t.numel() // t.shape[-1], t.shape[-1]
    if t.shape[-1] > 1 and t.numel() > 0 and t.stride(-1) != 1:
        raise ValueError(f"{name}: the last axis must be contiguous")
    rows, stride = 1, None
    for n, st in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if n > 1 and rows > 0:
            if stride is None:
                stride = st
            elif st != stride * rows:
                raise ValueError(f"{name}: the leading axes must be evenly spaced rows, got "
                                 f"strides {tuple(t.stride())}")
        rows *= n
    return rows, t.shape[-1] if stride is None else stride


def layer_norm(x, weight=None, bias=None, eps=1e-5, out=None, out_dtype=None, stats=None,
               stream=None):
    """Layer norm over the last axis: y = (x - mean) rstd weight + bias.

    x [..., D] fp32 or bf16 (evenly spaced rows), weight and bias [D] fp32 or None ->
    (y [..., D] of out_dtype (x's by default), mean [...], rstd [...] fp32, which
    ``layer_norm_backward`` reads).  out_dtype=torch.bfloat16 on a solve's fp32 h gives
    the next projection's input."""
    lib = load()
    dx = _norm_dtype("x", x)
    M, sx = _rows("x", x)
    D = x.shape[-1]
    _check_dev("weight", weight, torch.float32, (D,))
    _check_dev("bias", bias, torch.float32, (D,))
    if out_dtype is None:
        out_dtype = x.dtype if out is None else out.dtype
    if out_dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("out_dtype must be float32 or bfloat16")
    y, (mean, rstd) = out, stats or (None, None)
    with _making_on(stream):
        if out is None:
            y = torch.empty_like(x, dtype=out_dtype, memory_format=torch.contiguous_format)
        if stats is None:
            mean = x.new_empty(x.shape[:-1], dtype=torch.float32)
            rstd = torch.empty_like(mean)
    if out is None and stats is None:
        dev = _one_device(x=x, weight=weight, bias=bias)
    else:
        _check_dev("out", y, out_dtype, x.shape)
        _check_dev("mean", mean, torch.float32, x.shape[:-1])
        _check_dev("rstd", rstd, torch.float32, x.shape[:-1])
        dev = _one_device(x=x, weight=weight, bias=bias, out=y, mean=mean, rstd=rstd)
        _apart((("out", y), ("mean", mean), ("rstd", rstd)),
               (("x", x), ("weight", weight), ("bias", bias)))
    with _device_guard(dev):
        st = lib.pararnn_layer_norm(_ptr(x), dx, sx, _ptr(weight), _ptr(bias), _ptr(y),
                                    BF16 if out_dtype == torch.bfloat16 else F32, _ptr(mean),
                                    _ptr(rstd), M, D, float(eps), _stream_handle(stream, dev))
    _raise(st, "pararnn_layer_norm")
    return y, mean, rstd


def layer_norm_backward(dy, x, mean, rstd, weight=None, out=None, stream=None):
    """Gradients of a loss through ``layer_norm``, given dy = dl/dy (fp32 or bf16, x's
    shape) and the mean and rstd it returned: (dx of x's type, dweight [D], dbias [D]
    fp32).  The weight's gradient is summed in a fixed order."""
    lib = load()
    tx, ty = _norm_dtype("x", x), _norm_dtype("dy", dy)
    M, sx = _rows("x", x)
    if tuple(dy.shape) != tuple(x.shape):
        raise ValueError(f"dy: expected shape {tuple(x.shape)}, got {tuple(dy.shape)}")
    _, sdy = _rows("dy", dy)
    D, lead = x.shape[-1], x.shape[:-1]
    _check_dev("weight", weight, torch.float32, (D,))
    _check_dev("mean", mean, torch.float32, lead)
    _check_dev("rstd", rstd, torch.float32, lead)
    if out is None:
        with _making_on(stream):
            dx = torch.empty_like(x, memory_format=torch.contiguous_format)
            dw, db = mean.new_empty(D), mean.new_empty(D)
        dev = _one_device(dy=dy, x=x, mean=mean, rstd=rstd, weight=weight)
    else:
        dx, dw, db = out
        _check_dev("dx", dx, x.dtype, x.shape)
        _check_dev("dweight", dw, torch.float32, (D,))
        _check_dev("dbias", db, torch.float32, (D,))
        dev = _one_device(dy=dy, x=x, mean=mean, rstd=rstd, weight=weight, dx=dx, dweight=dw,
                          dbias=db)
        _apart((("dx", dx), ("dweight", dw), ("dbias", db)),
               (("dy", dy), ("x", x), ("mean", mean), ("rstd", rstd), ("weight", weight)))
    nws = lib.pararnn_layer_norm_workspace_size(M, D)
    ws = _call_buffer(nws, dev, stream)
    with _device_guard(dev):
        st = lib.pararnn_layer_norm_backward(_ptr(dy), ty, sdy, _ptr(x), tx, sx, _ptr(weight),
                                             _ptr(mean), _ptr(rstd), _ptr(dx), _ptr(dw),
                                             _ptr(db), M, D, _ptr(ws), nws,
                                             _stream_handle(stream, dev))
    _raise(st, "pararnn_layer_norm_backward")
    return dx, dw, db


PROBE_MUFU, PROBE_FMA = 0, 1


def probe_rate(pipe, iters, sink, stream=None):
    """Enqueue one throughput-probe launch (``pararnn_probe_rate``) and return
    the number of operations it performs: ex2 + rcp for ``PROBE_MUFU``, FMAs
    for ``PROBE_FMA``.  ``sink`` is a device tensor of at least 4 bytes."""
    lib = load()
    if not sink.is_cuda or sink.numel() * sink.element_size() < 4:
        raise ValueError("sink must be a CUDA tensor of at least 4 bytes")
    ops = ctypes.c_int64(0)
    with _device_guard(sink.device):
        st = lib.pararnn_probe_rate(int(pipe), int(iters), _ptr(sink), ctypes.byref(ops),
                                    _stream_handle(stream, sink.device))
    _raise(st, "pararnn_probe_rate")
    return int(ops.value)

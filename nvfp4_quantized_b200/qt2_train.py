"""Thin ctypes binding of the training operators' C ABI (include/qt2_train.h): layer norm, the
head's softmax cross entropy and the global gradient norm with clipping, in ``libqt2_train.so``.

Argument marshalling only, in the manner of ``qt2``: every function forwards to the entry point of
the same name with the tensors' device pointers and the current CUDA stream (or ``stream``), and
raises ``QT2Error`` on a non-OK status.  Element types are the tensors' own (bf16 or fp32); before
the call a tensor that is not on the current CUDA device raises ``QT2Error`` with QT2_ERR_DEVICE, one
of a type that the call does not take with QT2_ERR_INVALID_ARG, as does a vector (weights, statistics,
targets, losses and their gradients, workspaces) that is not contiguous: an expanded or strided one
holds other elements, or fewer, than the call reads.  Matrices are given by their leading dimension.
There is no fallback.
"""
from __future__ import annotations

import array
import ctypes
import os
import re
import threading

import torch

from . import qt2
from .qt2 import QT2_DTYPE_BF16, QT2_DTYPE_F32, QT2_ERR_DEVICE, QT2_ERR_INVALID_ARG, FaultHookC, QT2Error

_PKG = os.path.dirname(os.path.abspath(__file__))
# QT2_LIBRARY=checked loads the checked build, as in qt2
LIB_PATH = os.path.join(_PKG, "libqt2_train_checked.so" if os.environ.get("QT2_LIBRARY") == "checked"
                        else "libqt2_train.so")
HEADER_PATH = os.path.join(os.path.dirname(_PKG), "include", "qt2_train.h")

_DTYPE = {torch.bfloat16: QT2_DTYPE_BF16, torch.float32: QT2_DTYPE_F32}


class GradC(ctypes.Structure):
    _fields_ = [("grad", ctypes.c_void_p), ("out", ctypes.c_void_p), ("numel", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


_lock = threading.Lock()
_lib = None


def lib() -> ctypes.CDLL:
    """Load libqt2_train.so (built in-tree by nvfp4_quantized_b200.build); raise if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m nvfp4_quantized_b200.build` "
                                   "(there is no fallback path)")
            L = ctypes.CDLL(LIB_PATH)
            i32, i64, sz, vp, f32 = ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_float
            psz = ctypes.POINTER(ctypes.c_size_t)
            sigs = {
                "qt2_train_device_status": (i32, [vp, ctypes.POINTER(ctypes.c_int)]),
                "qt2_train_set_fault_hook": (None, [FaultHookC, vp]),
                "qt2_train_build_checked": (i32, []),
                "qt2_layernorm_fwd": (i32, [vp, i32, i64, i64, i64, vp, vp, i32, f32, vp, i64, vp, vp, vp]),
                "qt2_layernorm_bwd_workspace_size": (i32, [i64, i64, psz]),
                "qt2_layernorm_bwd": (i32, [vp, i64, vp, i32, i64, i64, i64, vp, i32, vp, vp, vp, i64, vp, vp, vp, sz,
                                            vp]),
                "qt2_linear_xent_fwd_workspace_size": (i32, [i64, i64, i64, psz]),
                "qt2_linear_xent_fwd": (i32, [vp, vp, vp, i64, i64, i64, i64, i64, i64, vp, vp, vp, sz, vp]),
                "qt2_linear_xent_bwd_workspace_size": (i32, [i64, i64, i64, psz]),
                "qt2_linear_xent_bwd": (i32, [vp, vp, vp, vp, vp, i64, i64, i64, i64, i64, i64, vp, i64, vp, i32, i64,
                                              vp, sz, vp]),
                "qt2_grad_norm_workspace_size": (i32, [vp, i64, psz]),
                "qt2_grad_norm": (i32, [vp, i64, vp, vp, sz, vp]),
                "qt2_grad_clip": (i32, [vp, i64, vp, f32, vp]),
            }
            for name, (res, args) in sigs.items():
                fn = getattr(L, name)
                fn.restype = res
                fn.argtypes = args
            _lib = L
    return _lib


def header_functions() -> list[str]:
    """Names of the functions include/qt2_train.h declares."""
    text = re.sub(r"/\*.*?\*/", "", open(HEADER_PATH).read(), flags=re.S)
    return sorted(set(re.findall(r"QT2_API\s+\w+\s+(qt2_[A-Za-z0-9_]+)\s*\(", text)))


def _check(fn: str, status: int):
    if status != 0:
        raise QT2Error(fn, status)


def _ptrs(fn: str, *tensors):
    """Device pointers of tensors (None stays None); all of them on the current device."""
    dev = torch.cuda.current_device()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise QT2Error(fn, QT2_ERR_DEVICE)
    return [None if t is None else t.data_ptr() for t in tensors]


def _dtype(fn: str, *tensors) -> int:
    """The common element type of tensors (None is skipped); QT2_DTYPE_BF16 if there is none."""
    found = None
    for t in tensors:
        if t is None or t.dtype is found:
            continue
        if found is not None or t.dtype not in _DTYPE:
            raise QT2Error(fn, QT2_ERR_INVALID_ARG)
        found = t.dtype
    return QT2_DTYPE_BF16 if found is None else _DTYPE[found]


def _only(fn: str, dtype: torch.dtype, *tensors):
    for t in tensors:
        if t is not None and t.dtype is not dtype:
            raise QT2Error(fn, QT2_ERR_INVALID_ARG)


def _vectors(fn: str, *tensors):
    for t in tensors:
        if t is not None and not t.is_contiguous():
            raise QT2Error(fn, QT2_ERR_INVALID_ARG)


# The current stream's handle; torch.cuda.current_stream() makes a Stream object for it, which takes
# longer than a small kernel (3.4 us).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> int:
    if stream is None and _raw_stream is not None:
        return _raw_stream(torch.cuda.current_device())
    return qt2._stream(stream)


# --------------------------------------------------------------------------------------------- entry points
def qt2_train_device_status(stream=None) -> int:
    code = ctypes.c_int(0)
    _check("qt2_train_device_status", lib().qt2_train_device_status(_stream(stream), ctypes.byref(code)))
    return code.value


def qt2_train_build_checked() -> bool:
    """True when the loaded library is the checked build (QT2_LIBRARY=checked)."""
    return bool(lib().qt2_train_build_checked())


def qt2_layernorm_fwd(x: torch.Tensor, rows: int, cols: int, ldx: int, weight: torch.Tensor | None,
                      bias: torch.Tensor | None, eps: float, y: torch.Tensor, ldy: int, mean: torch.Tensor | None,
                      rstd: torch.Tensor | None, stream=None) -> None:
    """y = (x - mean) * rstd * weight + bias over the rows of x; x and y of one type, weight and
    bias of one type, mean and rstd fp32."""
    fn = "qt2_layernorm_fwd"
    xd, wd = _dtype(fn, x, y), _dtype(fn, weight, bias)
    _only(fn, torch.float32, mean, rstd)
    _vectors(fn, weight, bias, mean, rstd)
    px, pw, pb, py, pm, pr = _ptrs(fn, x, weight, bias, y, mean, rstd)
    _check(fn, lib().qt2_layernorm_fwd(px, xd, rows, cols, ldx, pw, pb, wd, eps, py, ldy, pm, pr, _stream(stream)))


def qt2_layernorm_bwd_workspace_size(rows: int, cols: int) -> int:
    n = ctypes.c_size_t(0)
    _check("qt2_layernorm_bwd_workspace_size", lib().qt2_layernorm_bwd_workspace_size(rows, cols, ctypes.byref(n)))
    return n.value


def qt2_layernorm_bwd(dy: torch.Tensor, lddy: int, x: torch.Tensor, rows: int, cols: int, ldx: int,
                      weight: torch.Tensor | None, mean: torch.Tensor, rstd: torch.Tensor, dx: torch.Tensor | None,
                      lddx: int, dweight: torch.Tensor | None, dbias: torch.Tensor | None, workspace: torch.Tensor,
                      ws_bytes: int, stream=None) -> None:
    """dx, dweight and dbias (each may be None, not all) of qt2_layernorm_fwd; dy, x and dx of one
    type, weight, dweight and dbias of one type."""
    fn = "qt2_layernorm_bwd"
    xd, wd = _dtype(fn, dy, x, dx), _dtype(fn, weight, dweight, dbias)
    _only(fn, torch.float32, mean, rstd)
    _vectors(fn, weight, mean, rstd, dweight, dbias, workspace)
    pdy, px, pw, pm, pr, pdx, pdw, pdb, pws = _ptrs(fn, dy, x, weight, mean, rstd, dx, dweight, dbias, workspace)
    _check(fn, lib().qt2_layernorm_bwd(pdy, lddy, px, xd, rows, cols, ldx, pw, wd, pm, pr, pdx, lddx, pdw, pdb, pws,
                                       ws_bytes, _stream(stream)))


def qt2_linear_xent_fwd_workspace_size(T: int, K: int, V: int) -> int:
    n = ctypes.c_size_t(0)
    _check("qt2_linear_xent_fwd_workspace_size", lib().qt2_linear_xent_fwd_workspace_size(T, K, V, ctypes.byref(n)))
    return n.value


def qt2_linear_xent_fwd(x: torch.Tensor, w: torch.Tensor, targets: torch.Tensor, T: int, K: int, V: int, ldx: int,
                        ldw: int, ignore_index: int, loss: torch.Tensor, lse: torch.Tensor, workspace: torch.Tensor,
                        ws_bytes: int, stream=None) -> None:
    """Softmax cross entropy of the logits x w^T (x [T, K], w [V, K] bf16) against int64 targets:
    loss and lse [T] fp32; the logits are never stored."""
    fn = "qt2_linear_xent_fwd"
    _only(fn, torch.bfloat16, x, w)
    _only(fn, torch.int64, targets)
    _only(fn, torch.float32, loss, lse)
    _vectors(fn, targets, loss, lse, workspace)
    px, pw, pt, pl, ps, pws = _ptrs(fn, x, w, targets, loss, lse, workspace)
    _check(fn, lib().qt2_linear_xent_fwd(px, pw, pt, T, K, V, ldx, ldw, ignore_index, pl, ps, pws, ws_bytes,
                                         _stream(stream)))


def qt2_linear_xent_bwd_workspace_size(T: int, K: int, V: int) -> int:
    n = ctypes.c_size_t(0)
    _check("qt2_linear_xent_bwd_workspace_size", lib().qt2_linear_xent_bwd_workspace_size(T, K, V, ctypes.byref(n)))
    return n.value


def qt2_linear_xent_bwd(x: torch.Tensor, w: torch.Tensor, targets: torch.Tensor, lse: torch.Tensor,
                        dloss: torch.Tensor, T: int, K: int, V: int, ldx: int, ldw: int, ignore_index: int,
                        dx: torch.Tensor | None, lddx: int, dw: torch.Tensor | None, dw_dtype: int, lddw: int,
                        workspace: torch.Tensor, ws_bytes: int, stream=None) -> None:
    """dx [T, K] bf16 and dw [V, K] of type dw_dtype (either may be None) of sum(dloss * loss)."""
    fn = "qt2_linear_xent_bwd"
    _only(fn, torch.bfloat16, x, w, dx)
    _only(fn, torch.int64, targets)
    _only(fn, torch.float32, lse, dloss)
    _vectors(fn, targets, lse, dloss, workspace)
    if dw is not None and _dtype(fn, dw) != dw_dtype:
        raise QT2Error(fn, QT2_ERR_INVALID_ARG)
    px, pw, pt, ps, pg, pdx, pdw, pws = _ptrs(fn, x, w, targets, lse, dloss, dx, dw, workspace)
    _check(fn, lib().qt2_linear_xent_bwd(px, pw, pt, ps, pg, T, K, V, ldx, ldw, ignore_index, pdx, lddx, pdw, dw_dtype,
                                         lddw, pws, ws_bytes, _stream(stream)))


class GradList:
    """The list that qt2_grad_norm and qt2_grad_clip take: contiguous bf16 or fp32 tensors on one
    device, and where each one's clipped gradient goes (`outs`; None: in place).  Made once for
    buffers that stay where they are; it keeps the tensors alive."""

    def __init__(self, grads, outs=None):
        fn = "GradList"
        self.grads = list(grads)
        self.outs = self.grads if outs is None else list(outs)
        self.count = n = len(self.grads)
        both = self.grads if outs is None else self.grads + self.outs
        kinds = [_DTYPE.get(t.dtype) for t in both]
        if len(self.outs) != n or None in kinds or not all([t.is_contiguous() for t in both]):
            raise QT2Error(fn, QT2_ERR_INVALID_ARG)
        devices = {t.get_device() for t in both}
        if len(devices) > 1:
            raise QT2Error(fn, QT2_ERR_DEVICE)
        self.device = devices.pop() if devices else -1
        at, numel = [t.data_ptr() for t in both], [t.numel() for t in both]
        out = 0 if outs is None else n   # where the outputs begin
        if numel[:n] != numel[out:] or kinds[:n] != kinds[out:]:
            raise QT2Error(fn, QT2_ERR_INVALID_ARG)
        # what one entry writes and another reads or writes too has no one value
        spans = [(p, p + m * (4 if k else 2), 1) for p, m, k in zip(at[out:], numel, kinds) if m]
        if out:
            spans += [(p, p + m * (4 if k else 2), 0) for p, q, m, k in zip(at, at[n:], numel, kinds) if m and p != q]
        spans.sort()
        written = read = 0   # ends of what has been seen
        for lo, hi, writes in spans:
            if lo < written or (writes and lo < read):
                raise QT2Error(fn, QT2_ERR_INVALID_ARG)
            if writes:
                written = hi
            elif hi > read:
                read = hi
        rows = array.array("q", [v for row in zip(at[:n], at[out:], numel, kinds) for v in row] or [0] * 4)
        self.c = (GradC * max(1, n)).from_buffer(rows)   # the type is the lower half of the last number
        self.address = ctypes.addressof(self.c)


def qt2_grad_norm_workspace_size(grads: GradList) -> int:
    n = ctypes.c_size_t(0)
    _check("qt2_grad_norm_workspace_size",
           lib().qt2_grad_norm_workspace_size(grads.address, grads.count, ctypes.byref(n)))
    return n.value


def qt2_grad_norm(grads: GradList, norm: torch.Tensor, workspace: torch.Tensor, ws_bytes: int, stream=None) -> None:
    """norm (one fp32 element) = the 2-norm of all the list's gradients together."""
    fn = "qt2_grad_norm"
    _only(fn, torch.float32, norm)
    _vectors(fn, workspace)
    pn, pws = _ptrs(fn, norm, workspace)
    if grads.count and grads.device != norm.get_device():
        raise QT2Error(fn, QT2_ERR_DEVICE)
    _check(fn, lib().qt2_grad_norm(grads.address, grads.count, pn, pws, ws_bytes, _stream(stream)))


def qt2_grad_clip(grads: GradList, norm: torch.Tensor, max_norm: float, stream=None) -> None:
    """Every gradient times min(1, max_norm / (norm + 1e-6)) into its `out`."""
    fn = "qt2_grad_clip"
    _only(fn, torch.float32, norm)
    pn, = _ptrs(fn, norm)
    if grads.count and grads.device != norm.get_device():
        raise QT2Error(fn, QT2_ERR_DEVICE)
    _check(fn, lib().qt2_grad_clip(grads.address, grads.count, pn, max_norm, _stream(stream)))


class fault_hook(qt2.fault_hook):
    """qt2.fault_hook around qt2_train_set_fault_hook."""

    def __enter__(self):
        lib().qt2_train_set_fault_hook(self._c, None)
        return self

    def __exit__(self, *exc):
        lib().qt2_train_set_fault_hook(FaultHookC(), None)
        return False

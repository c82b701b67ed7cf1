"""Thin ctypes binding of the training operators' C ABI (include/qt2_train.h): layer norm, the
head's softmax cross entropy, the gated feed-forward product on NVFP4 operands, the norm of queries and
keys with the position rotation, the global gradient norm with clipping and the AdamW step of many
tensors, in ``libqt2_train.so``.

Argument marshalling only, in the manner of ``qt2``: every function forwards to the entry point of
the same name with the tensors' device pointers and the current CUDA stream (or ``stream``), and
raises ``QT2Error`` on a non-OK status.  Element types are the tensors' own (bf16 or fp32); before
the call a tensor that is not on the current CUDA device raises ``QT2Error`` with QT2_ERR_DEVICE, one
of a type that the call does not take with QT2_ERR_INVALID_ARG, as does a vector (weights, statistics,
targets, losses and their gradients, workspaces) that is not contiguous: an expanded or strided one
holds other elements, or fewer, than the call reads.  Matrices are given by their leading dimension.
Views, and the weights, positions and tables of the norm of queries and keys, that do not have the sizes of the
call raise it with QT2_ERR_SHAPE.
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
from .qt2 import (QT2_DTYPE_BF16, QT2_DTYPE_F32, QT2_ERR_DEVICE, QT2_ERR_INVALID_ARG, QT2_ERR_SHAPE, FaultHookC,
                  QT2Error)

_PKG = os.path.dirname(os.path.abspath(__file__))
# QT2_LIBRARY=checked loads the checked build, as in qt2
LIB_PATH = os.path.join(_PKG, "libqt2_train_checked.so" if os.environ.get("QT2_LIBRARY") == "checked"
                        else "libqt2_train.so")
HEADER_PATH = os.path.join(os.path.dirname(_PKG), "include", "qt2_train.h")

QT2_ACT_SILU, QT2_ACT_GELU_TANH = 0, 1
QT2_ROPE_HALVES, QT2_ROPE_PAIRS = 0, 1
QT2_STATE_F32, QT2_STATE_E4M3 = 0, 1

_DTYPE = {torch.bfloat16: QT2_DTYPE_BF16, torch.float32: QT2_DTYPE_F32}
_STATE = {torch.float32: QT2_STATE_F32, torch.float8_e4m3fn: QT2_STATE_E4M3}


class GradC(ctypes.Structure):
    _fields_ = [("grad", ctypes.c_void_p), ("out", ctypes.c_void_p), ("numel", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class AdamWTensorC(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("param", "master", "grad", "m", "v", "m_scale", "v_scale")] + [
        ("numel", ctypes.c_int64), ("param_dtype", ctypes.c_int32), ("grad_dtype", ctypes.c_int32),
        ("state", ctypes.c_int32), ("weight_decay", ctypes.c_float)]


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
            psz, pv = ctypes.POINTER(ctypes.c_size_t), ctypes.POINTER(qt2.NVFP4ViewC)
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
                "qt2_gemm_nvfp4_gated": (i32, [pv, pv, pv, i64, i64, i64, f32, i32, vp, vp, i64, vp, i64, vp]),
                "qt2_gemm_nvfp4_gated_bwd": (i32, [pv, pv, i64, i64, i64, f32, i32, vp, vp, i64, vp, vp, i64, vp, i64,
                                                   vp]),
                "qt2_qk_norm_rope_fwd": (i32, [vp, i32, i64, i64, i64, i64, i64, i64, vp, vp, i32, f32, vp, vp, vp, i64,
                                               i64, i32, vp, i64, i64, vp]),
                "qt2_qk_norm_rope_bwd_workspace_size": (i32, [i64, i64, i64, i64, psz]),
                "qt2_qk_norm_rope_bwd": (i32, [vp, i64, i64, vp, i32, i64, i64, i64, i64, i64, i64, vp, vp, i32, f32, vp,
                                               vp, vp, i64, i64, i32, vp, i64, i64, vp, vp, vp, sz, vp]),
                "qt2_grad_norm_workspace_size": (i32, [vp, i64, psz]),
                "qt2_grad_norm": (i32, [vp, i64, vp, vp, sz, vp]),
                "qt2_grad_clip": (i32, [vp, i64, vp, f32, vp]),
                "qt2_adamw": (i32, [vp, i64, vp, vp, ctypes.c_double, ctypes.c_double, f32, vp, f32, ctypes.c_uint64, vp]),
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
    found = []
    for t in tensors:
        if t is None:
            found.append(None)
            continue
        if t.get_device() != dev:
            raise QT2Error(fn, QT2_ERR_DEVICE)
        found.append(t.data_ptr())
    return found


def _dtype(fn: str, *tensors) -> int:
    """The common element type of tensors (None is skipped); QT2_DTYPE_BF16 if there is none."""
    found = None
    for t in tensors:
        if t is not None:
            d = t.dtype
            if d is not found:
                if found is not None or d not in _DTYPE:
                    raise QT2Error(fn, QT2_ERR_INVALID_ARG)
                found = d
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


def _stream(stream, device: int | None = None) -> int:
    """`device`: the current one, where the caller knows it (its tensors were found to be on it)."""
    if stream is None and _raw_stream is not None:
        return _raw_stream(torch.cuda.current_device() if device is None else device)
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


def _view(fn: str, v: qt2.View, R: int, C: int):
    """The arrays of an [R, C] view."""
    codes, scales, scale = v.codes, v.scales, v.tensor_scale
    if (codes.dtype is not torch.uint8 or scales.dtype is not torch.uint8 or scale.dtype is not torch.float32
            or not codes.is_contiguous() or not scales.is_contiguous()):
        raise QT2Error(fn, QT2_ERR_INVALID_ARG)
    # a view of other sizes holds fewer elements than the call reads, or others (sizes that no call takes are its to refuse)
    if R > 0 and C > 0 and (codes.numel() != R * C // 2 or scales.numel() != R * C // 16):
        raise QT2Error(fn, QT2_ERR_SHAPE)
    # of the scales of a view with one for 128 rows, which differs from this one in nothing else, all but the first
    # would be left out
    if scale.numel() != 1:
        raise QT2Error(fn, QT2_ERR_SHAPE)
    return codes, scales, scale


def qt2_gemm_nvfp4_gated(a: qt2.View, b_gate: qt2.View, b_up: qt2.View, M: int, F: int, K: int, alpha: float, act: int,
                         gate: torch.Tensor | None, up: torch.Tensor | None, ldgu: int, h: torch.Tensor, ldh: int,
                         stream=None) -> None:
    """h = act(g) * u of the two products g = alpha a b_gate^T and u = alpha a b_up^T (views [M, K], [F, K],
    [F, K]); g and u go to gate and up (for the backward pass; None: not kept).  bf16 outputs."""
    fn = "qt2_gemm_nvfp4_gated"
    _only(fn, torch.bfloat16, gate, up, h)
    p = _ptrs(fn, *_view(fn, a, M, K), *_view(fn, b_gate, F, K), *_view(fn, b_up, F, K), gate, up, h)
    va, vg, vu = qt2.NVFP4ViewC(*p[:3]), qt2.NVFP4ViewC(*p[3:6]), qt2.NVFP4ViewC(*p[6:9])
    _check(fn, lib().qt2_gemm_nvfp4_gated(va, vg, vu, M, F, K, alpha, act, p[9], p[10], ldgu, p[11], ldh,
                                          _stream(stream, h.get_device())))


def qt2_gemm_nvfp4_gated_bwd(a: qt2.View, b: qt2.View, M: int, F: int, K: int, alpha: float, act: int,
                             gate: torch.Tensor, up: torch.Tensor, ldgu: int, dgate: torch.Tensor, dup: torch.Tensor,
                             lddgu: int, h: torch.Tensor | None, ldh: int, stream=None) -> None:
    """dgate = dh up act'(gate), dup = dh act(gate) and h = act(gate) up (None: not wanted) of
    dh = alpha a b^T (views [M, K], [F, K]), which is not stored.  bf16 outputs."""
    fn = "qt2_gemm_nvfp4_gated_bwd"
    _only(fn, torch.bfloat16, gate, up, dgate, dup, h)
    p = _ptrs(fn, *_view(fn, a, M, K), *_view(fn, b, F, K), gate, up, dgate, dup, h)
    va, vb = qt2.NVFP4ViewC(*p[:3]), qt2.NVFP4ViewC(*p[3:6])
    _check(fn, lib().qt2_gemm_nvfp4_gated_bwd(va, vb, M, F, K, alpha, act, p[6], p[7], ldgu, p[8], p[9], lddgu, p[10],
                                              ldh, _stream(stream, gate.get_device())))


def _qk_vectors(fn: str, T: int, D: int, P: int, R: int, positions, cos, sin, *weights):
    """Contiguous weights of D elements, an int64 position for each token, fp32 tables of [P, R/2] or of more such
    rows (sizes that no call takes are its to refuse).  One function: the checks of a small call are part of its time."""
    status = 0
    for w in weights:
        if w is not None:
            if not w.is_contiguous():
                raise QT2Error(fn, QT2_ERR_INVALID_ARG)
            if w.numel() != D > 0:
                status = QT2_ERR_SHAPE
    if positions is not None:
        if positions.dtype is not torch.int64 or not positions.is_contiguous():
            raise QT2Error(fn, QT2_ERR_INVALID_ARG)
        if positions.numel() < T:
            status = QT2_ERR_SHAPE
    n = P * (R // 2)
    for t in (cos, sin):
        if t is not None:
            if t.dtype is not torch.float32 or not t.is_contiguous():
                raise QT2Error(fn, QT2_ERR_INVALID_ARG)
            # more elements are more rows, or rows that hold an angle twice
            if t.numel() != n > 0 and (t.numel() < n or t.dim() < 2 or t.shape[-1] != R // 2):
                status = QT2_ERR_SHAPE
    if status:
        raise QT2Error(fn, status)


def qt2_qk_norm_rope_fwd(x: torch.Tensor, T: int, Hq: int, Hk: int, D: int, ldx: int, hsx: int,
                         wq: torch.Tensor | None, wk: torch.Tensor | None, eps: float, positions: torch.Tensor | None,
                         cos: torch.Tensor | None, sin: torch.Tensor | None, P: int, R: int, pairing: int,
                         y: torch.Tensor, ldy: int, hsy: int, stream=None) -> None:
    """y = the Hq + Hk heads of x, each divided by its root mean square, times wq or wk, its first R elements
    turned by row positions[t] of the tables cos and sin [P, R/2].  x and y of one type, wq and wk of one type."""
    fn = "qt2_qk_norm_rope_fwd"
    xd, wd = _dtype(fn, x, y), _dtype(fn, wq, wk)
    _qk_vectors(fn, T, D, P, R, positions, cos, sin, wq, wk)
    px, pq, pk, pp, pc, ps, py = _ptrs(fn, x, wq, wk, positions, cos, sin, y)
    _check(fn, lib().qt2_qk_norm_rope_fwd(px, xd, T, Hq, Hk, D, ldx, hsx, pq, pk, wd, eps, pp, pc, ps, P, R, pairing, py,
                                          ldy, hsy, _stream(stream, x.get_device())))


def qt2_qk_norm_rope_bwd_workspace_size(T: int, Hq: int, Hk: int, D: int) -> int:
    n = ctypes.c_size_t(0)
    _check("qt2_qk_norm_rope_bwd_workspace_size",
           lib().qt2_qk_norm_rope_bwd_workspace_size(T, Hq, Hk, D, ctypes.byref(n)))
    return n.value


def qt2_qk_norm_rope_bwd(dy: torch.Tensor, lddy: int, hsdy: int, x: torch.Tensor, T: int, Hq: int, Hk: int, D: int,
                         ldx: int, hsx: int, wq: torch.Tensor | None, wk: torch.Tensor | None, eps: float,
                         positions: torch.Tensor | None, cos: torch.Tensor | None, sin: torch.Tensor | None, P: int,
                         R: int, pairing: int, dx: torch.Tensor | None, lddx: int, hsdx: int,
                         dwq: torch.Tensor | None, dwk: torch.Tensor | None, workspace: torch.Tensor, ws_bytes: int,
                         stream=None) -> None:
    """dx, dwq and dwk (each may be None, not all) of qt2_qk_norm_rope_fwd; dy, x and dx of one type, wq, wk,
    dwq and dwk of one type."""
    fn = "qt2_qk_norm_rope_bwd"
    xd, wd = _dtype(fn, dy, x, dx), _dtype(fn, wq, wk, dwq, dwk)
    _vectors(fn, workspace)
    _qk_vectors(fn, T, D, P, R, positions, cos, sin, wq, wk, dwq, dwk)
    pdy, px, pq, pk, pp, pc, ps, pdx, pdq, pdk, pws = _ptrs(fn, dy, x, wq, wk, positions, cos, sin, dx, dwq, dwk,
                                                            workspace)
    _check(fn, lib().qt2_qk_norm_rope_bwd(pdy, lddy, hsdy, px, xd, T, Hq, Hk, D, ldx, hsx, pq, pk, wd, eps, pp, pc, ps, P,
                                          R, pairing, pdx, lddx, hsdx, pdq, pdk, pws, ws_bytes, _stream(stream, x.get_device())))


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


class AdamWList:
    """The list that qt2_adamw takes: parameters (bf16 or fp32), their gradients (bf16 or fp32) and states m and v,
    contiguous tensors on one device.  States are fp32, or torch.float8_e4m3fn with fp32 scales of one element for
    256 in m_scales and v_scales.  masters: an fp32 tensor for each bf16 parameter, or None (no masters), in the
    whole list's place or an entry's.  weight_decay: one number, or one for each.  Made once for buffers that stay
    where they are (gradients too: zeroed, not set to None; making it takes 1.1 ms for 300 tensors); it keeps the
    tensors alive."""

    def __init__(self, params, grads, m, v, masters=None, m_scales=None, v_scales=None, weight_decay=0.0):
        fn = "AdamWList"
        self.params, self.grads, self.m, self.v = (list(t) for t in (params, grads, m, v))
        self.count = n = len(self.params)
        self.masters, self.m_scales, self.v_scales = ([None] * n if t is None else list(t)
                                                      for t in (masters, m_scales, v_scales))
        decay = [float(weight_decay)] * n if isinstance(weight_decay, (int, float)) else [float(w) for w in weight_decay]
        columns = (self.params, self.masters, self.grads, self.m, self.v, self.m_scales, self.v_scales)
        if any(len(c) != n for c in columns) or len(decay) != n:
            raise QT2Error(fn, QT2_ERR_INVALID_ARG)
        kinds = [_DTYPE.get(t.dtype) for t in self.params], [_DTYPE.get(t.dtype) for t in self.grads]
        state = [_STATE.get(t.dtype) for t in self.m]
        if None in kinds[0] or None in kinds[1] or None in state or [_STATE.get(t.dtype) for t in self.v] != state:
            raise QT2Error(fn, QT2_ERR_INVALID_ARG)
        fp32 = torch.float32
        if any([t is not None and (k or t.dtype is not fp32) for k, t in zip(kinds[0], self.masters)]) or any(
                [(t is not None) != e or (e and t.dtype is not fp32) for ts in columns[5:] for e, t in zip(state, ts)]):
            raise QT2Error(fn, QT2_ERR_INVALID_ARG)
        given = [[t for t in c if t is not None] for c in columns]
        if not all([t.is_contiguous() for c in given for t in c]):
            raise QT2Error(fn, QT2_ERR_INVALID_ARG)
        sizes = [t.numel() for t in self.params]
        four = [4 * m for m in sizes]
        scales = [4 * ((m + 255) // 256) for m in sizes]
        states = [m if e else 4 * m for e, m in zip(state, sizes)]
        # bytes of each array (what is not given is skipped)
        extent = [[m * (4 if k else 2) for k, m in zip(kinds[0], sizes)], four, [m * (4 if k else 2) for k, m in zip(kinds[1], sizes)],
                  states, states, scales, scales]
        if any([t is not None and t.nbytes != m for c, ms in zip(columns, extent) for t, m in zip(c, ms)]):
            raise QT2Error(fn, QT2_ERR_INVALID_ARG)
        devices = {t.get_device() for c in given for t in c}
        if len(devices) > 1:
            raise QT2Error(fn, QT2_ERR_DEVICE)
        self.device = devices.pop() if devices else -1
        at = [[0 if t is None else t.data_ptr() for t in c] for c in columns]
        # what is written overlaps nothing else
        spans = [(p, p + m, k != 2) for k, (ps, ms) in enumerate(zip(at, extent)) for p, m in zip(ps, ms) if p and m]
        spans.sort()
        end, end_written = 0, 0
        for lo, hi, writes in spans:
            if lo < end_written or (writes and lo < end):
                raise QT2Error(fn, QT2_ERR_INVALID_ARG)
            if hi > end:
                end = hi
            if writes:
                end_written = hi
        bits = array.array("I", array.array("f", decay).tobytes())
        rows = [(*row[:8], row[8] | row[9] << 32, row[10] | row[11] << 32) for row in zip(*at, sizes, *kinds, state, bits)]
        flat = array.array("Q", [v for row in rows for v in row] or [0] * 10)
        self.c = (AdamWTensorC * max(1, n)).from_buffer(flat)
        self.address = ctypes.addressof(self.c)


def qt2_adamw(tensors: AdamWList, lr: torch.Tensor, step: torch.Tensor, beta1: float, beta2: float, eps: float,
              norm: torch.Tensor | None, max_norm: float, seed: int, stream=None) -> None:
    """One AdamW step of the list's tensors in place, gradients times min(1, max_norm / (norm + 1e-6)) (norm None:
    as they are).  lr (fp32), step (int64, from 1) and norm (fp32) are one element each on the device; seed draws
    the roundings of 8-bit states."""
    fn = "qt2_adamw"
    _only(fn, torch.float32, lr, norm)
    _only(fn, torch.int64, step)
    if any(t is not None and t.numel() != 1 for t in (lr, step, norm)):
        raise QT2Error(fn, QT2_ERR_INVALID_ARG)
    pl, ps, pn = _ptrs(fn, lr, step, norm)
    if tensors.count and tensors.device != lr.get_device():
        raise QT2Error(fn, QT2_ERR_DEVICE)
    _check(fn, lib().qt2_adamw(tensors.address, tensors.count, pl, ps, beta1, beta2, eps, pn, max_norm, seed,
                               _stream(stream, lr.get_device())))


class fault_hook(qt2.fault_hook):
    """qt2.fault_hook around qt2_train_set_fault_hook."""

    def __enter__(self):
        lib().qt2_train_set_fault_hook(self._c, None)
        return self

    def __exit__(self, *exc):
        lib().qt2_train_set_fault_hook(FaultHookC(), None)
        return False

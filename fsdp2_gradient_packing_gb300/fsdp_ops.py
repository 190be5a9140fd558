"""Thin ctypes binding of the training operators in include/fsdp_ops.h.

Each function has the name of the C entry point it calls.  Matrices are torch
tensors ``[rows, cols]`` with unit column stride and any row distance of at
least ``cols``; the binding takes their sizes and dtypes from the tensors,
checks them against one another (``ValueError``) and passes device pointers.
Where a call needs scratch and is given no ``workspace``, the binding takes one
from torch's caching allocator for the call.  Every call runs on the current
stream unless ``stream`` names another.

All names here are also names of ``fsdp_pack``.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import fsdp_pack as _fp
from .fsdp_pack import FSDP_DTYPE_BF16, FSDP_DTYPE_F32, _check, _current_stream, _lib

FSDP_ACT8 = 2
FSDP_ACT8_GROUP = 32
FSDP_NORM_MAX_COLS = 65536
FSDP_ACT_SILU, FSDP_ACT_GELU = 0, 1
FSDP_KEEP_NONE, FSDP_KEEP_ACT8, FSDP_KEEP_BF16 = 0, 1, 2

__all__ = ["FSDP_ACT8", "FSDP_ACT8_GROUP", "FSDP_NORM_MAX_COLS", "fsdp_norm_desc_t", "Act8", "fsdp_act8_bytes",
           "fsdp_act8_store", "fsdp_act8_load", "fsdp_layer_norm_forward", "fsdp_layer_norm_backward",
           "fsdp_layer_norm_workspace", "FSDP_ACT_SILU", "FSDP_ACT_GELU", "FSDP_KEEP_NONE", "FSDP_KEEP_ACT8",
           "FSDP_KEEP_BF16", "fsdp_ffn_desc_t", "fsdp_gated_ffn_forward", "fsdp_gated_ffn_backward",
           "fsdp_gated_ffn_workspace", "fsdp_ops_sync_status"]

_CODE = {torch.float32: FSDP_DTYPE_F32, torch.bfloat16: FSDP_DTYPE_BF16}


class fsdp_norm_desc_t(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("ld_x", ctypes.c_int64),
                ("ld_y", ctypes.c_int64), ("ld_dx", ctypes.c_int64), ("x_dtype", ctypes.c_int32),
                ("y_dtype", ctypes.c_int32), ("dx_dtype", ctypes.c_int32), ("param_dtype", ctypes.c_int32),
                ("grad_dtype", ctypes.c_int32), ("eps", ctypes.c_float)]


class fsdp_ffn_desc_t(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("rows", "d", "f", "ld_x", "ld_w_gate", "ld_w_up", "ld_h", "ld_kept",
                                              "ld_dx", "ld_dw_gate", "ld_dw_up")] + \
               [(n, ctypes.c_int32) for n in ("activation", "keep", "x_dtype", "dx_dtype", "dw_dtype", "unaligned")]


_P, _ST, _I64, _I32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_int32
_SIGNATURES = {
    "fsdp_act8_bytes": [_I64, _I64, ctypes.POINTER(_I64)],
    "fsdp_act8_store": [_P, _I32, _I64, _I64, _I64, _P, _P],
    "fsdp_act8_load": [_P, _I64, _I64, _P, _I32, _I64, _P],
    "fsdp_layer_norm_forward": [ctypes.POINTER(fsdp_norm_desc_t), _P, _P, _P, _P, _P, _P, _P, _P],
    "fsdp_layer_norm_backward": [ctypes.POINTER(fsdp_norm_desc_t), _P, _P, _P, _P, _P, _P, _P, _P, _P, _I64, _P],
    "fsdp_layer_norm_workspace": [ctypes.POINTER(fsdp_norm_desc_t), ctypes.POINTER(_I64)],
    "fsdp_gated_ffn_workspace": [ctypes.POINTER(fsdp_ffn_desc_t), _I32, ctypes.POINTER(_I64)],
    "fsdp_gated_ffn_forward": [ctypes.POINTER(fsdp_ffn_desc_t), _P, _P, _P, _P, _P, _P, _P, _I64, _P],
    "fsdp_gated_ffn_backward": [ctypes.POINTER(fsdp_ffn_desc_t)] + [_P] * 10 + [_I64, _P],
    "fsdp_ops_sync_status": [_P],
}
for _name, _args in _SIGNATURES.items():
    _fn = getattr(_lib, _name)
    _fn.restype = _ST
    _fn.argtypes = _args


# ---------------------------------------------------------------------------
# Arguments.  Each check takes and returns the device that the call's tensors are
# on (None before the first).  A small call costs little more on the GPU than
# these checks do on the host, so they are plain functions with few steps.
# ---------------------------------------------------------------------------
_BOTH, _BF16, _F32 = dict(_CODE), {torch.bfloat16: FSDP_DTYPE_BF16}, {torch.float32: FSDP_DTYPE_F32}
_get_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


@functools.lru_cache(maxsize=None)
def _device(index):
    return torch.device("cuda", index)


def _misplaced(where, what, index, device):
    if index < 0:
        raise ValueError(f"{where}: {what} is not a CUDA tensor")
    if device is not None:
        raise ValueError(f"{where}: {what} is on cuda:{index}, another argument on cuda:{device}")


def _matrix(where, what, t, rows, cols, codes, device):
    """(pointer, row distance, dtype code, device) of a [rows, cols] tensor; None: any size."""
    try:
        r, c = t.shape
        code = codes[t.dtype]
        s0, s1 = t.stride()
    except (AttributeError, TypeError, ValueError, KeyError):
        if not isinstance(t, torch.Tensor):
            raise ValueError(f"{where}: {what} is not a tensor") from None
        if t.dim() != 2:
            raise ValueError(f"{where}: {what} has {t.dim()} dimensions, not 2") from None
        raise ValueError(f"{where}: {what} is {t.dtype}, not one of {', '.join(map(str, codes))}") from None
    if (rows is not None and r != rows) or (cols is not None and c != cols):
        raise ValueError(f"{where}: {what} is {r} x {c}, not {r if rows is None else rows} x {c if cols is None else cols}")
    if s1 != 1 and c > 1:
        raise ValueError(f"{where}: {what} has column stride {s1}, not 1")
    if r <= 1 or s0 < c or c < 1:
        if c < 1:
            raise ValueError(f"{where}: {what} has no columns")
        if r > 1:
            raise ValueError(f"{where}: {what} has rows {s0} elements apart, fewer than its {c} columns")
        s0 = c
    index = t.get_device()
    if index != device:
        _misplaced(where, what, index, device)
    return t.data_ptr(), s0, code, index


def _vector(where, what, t, n, codes, device):
    """(pointer, dtype code, device) of a contiguous vector of n elements; no pointer or code for None."""
    if t is None:
        return None, None, device
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{where}: {what} is not a tensor")
    if t.numel() != n or not t.is_contiguous() or t.dim() > 1 and t.shape[-1] != n:
        raise ValueError(f"{where}: {what} is not a contiguous vector of {n} elements")
    code = codes.get(t.dtype)
    if code is None:
        raise ValueError(f"{where}: {what} is {t.dtype}, not one of {', '.join(map(str, codes))}")
    index = t.get_device()
    if index != device:
        _misplaced(where, what, index, device)
    return t.data_ptr(), code, index


def _ckpt(where, what, a, rows, cols, device):
    """(pointer, device) of the checkpoint of a [rows, cols] matrix."""
    if not isinstance(a, Act8):
        raise ValueError(f"{where}: {what} is not an Act8 checkpoint")
    if a.rows != rows or a.cols != cols:
        raise ValueError(f"{where}: {what} is a checkpoint of {a.rows} x {a.cols}, not of {rows} x {cols}")
    index = a.data.get_device()
    if index != device:
        _misplaced(where, what, index, device)
    return a.data.data_ptr(), index


def _handle(where, stream, device):
    """The handle of the stream to run on; the tensors have to be on the current device."""
    if device != _get_device():
        raise ValueError(f"{where}: the tensors are on cuda:{device}, the current device is {_get_device()}")
    if stream is None:
        return _current_stream()
    return stream if isinstance(stream, int) else stream.cuda_stream


def _workspace(where, given, nbytes, handle, device):
    """(pointer, bytes, owner) of the caller's workspace, or of one taken for this call."""
    if given is not None:
        if given.dtype != torch.uint8 or not given.is_contiguous():
            raise ValueError(f"{where}: workspace is not a contiguous uint8 tensor")
        if given.get_device() != device:
            _misplaced(where, "workspace", given.get_device(), device)
        if given.numel() < nbytes:
            raise ValueError(f"{where}: workspace holds {given.numel()} bytes, the call needs {nbytes}")
        return given.data_ptr(), given.numel(), given
    if nbytes == 0:
        return None, 0, None
    if handle == _current_stream():
        ws = torch.empty(nbytes, dtype=torch.uint8, device=_device(device))
    else:  # from the pool of the call's stream: what the current one gave back, its earlier launches may still be using
        other = torch.cuda.ExternalStream(handle, device=device) if handle else torch.cuda.default_stream(device)
        with torch.cuda.stream(other):
            ws = torch.empty(nbytes, dtype=torch.uint8, device=_device(device))
    return ws.data_ptr(), nbytes, ws


class Act8:
    """The 8-bit checkpoint of a ``[rows, cols]`` matrix: one uint8 tensor, codes ``[rows, 32 G]`` and then scale
    bytes ``[rows, G]`` with ``G = ceil(cols / 32)``.  ``data``: a buffer to use instead of a new one."""

    __slots__ = ("rows", "cols", "data")

    def __init__(self, rows, cols, data=None, device="cuda"):
        if rows < 0 or cols < 1:
            raise ValueError(f"Act8: no checkpoint of {rows} x {cols}")
        nbytes = rows * (FSDP_ACT8_GROUP + 1) * ((cols + FSDP_ACT8_GROUP - 1) // FSDP_ACT8_GROUP)
        if data is None:
            data = torch.empty(nbytes, dtype=torch.uint8, device=device)
        elif data.dtype != torch.uint8 or not data.is_contiguous() or data.numel() < nbytes:
            raise ValueError(f"Act8: data is not a contiguous uint8 tensor of at least {nbytes} bytes")
        self.rows, self.cols, self.data = rows, cols, data


def fsdp_act8_bytes(rows: int, cols: int) -> int:
    out = _I64()
    _check(_lib.fsdp_act8_bytes(rows, cols, ctypes.byref(out)), "fsdp_act8_bytes")
    return out.value


def fsdp_act8_store(x, ckpt: Act8, stream=None) -> None:
    where = "fsdp_act8_store"
    p, ld, dt, dev = _matrix(where, "x", x, None, None, _BOTH, None)
    c, dev = _ckpt(where, "ckpt", ckpt, *x.shape, dev)
    _check(_lib.fsdp_act8_store(p, dt, ckpt.rows, ckpt.cols, ld, c, _handle(where, stream, dev)), where)


def fsdp_act8_load(ckpt: Act8, y, stream=None) -> None:
    where = "fsdp_act8_load"
    p, ld, dt, dev = _matrix(where, "y", y, None, None, _BOTH, None)
    c, dev = _ckpt(where, "ckpt", ckpt, *y.shape, dev)
    _check(_lib.fsdp_act8_load(c, ckpt.rows, ckpt.cols, p, dt, ld, _handle(where, stream, dev)), where)


def _norm_input(where, x, rows, cols, dev):
    """(pointer, row distance, dtype code, device) of a norm's input, a tensor or a checkpoint."""
    if isinstance(x, Act8):
        p, dev = _ckpt(where, "x", x, rows, cols, dev)
        return p, cols, FSDP_ACT8, dev
    return _matrix(where, "x", x, rows, cols, _BOTH, dev)


def fsdp_layer_norm_forward(x, weight, bias, y, mean=None, rstd=None, eps=1e-5, keep=None, stream=None) -> None:
    """x: a tensor or its ``Act8`` checkpoint; keep: an ``Act8`` that receives x's checkpoint in the same pass."""
    where = "fsdp_layer_norm_forward"
    py, ld_y, dt_y, dev = _matrix(where, "y", y, None, None, _BOTH, None)
    rows, cols = y.shape
    px, ld_x, dt_x, dev = _norm_input(where, x, rows, cols, dev)
    pw, dt_w, dev = _vector(where, "weight", weight, cols, _BOTH, dev)
    pb, dt_b, dev = _vector(where, "bias", bias, cols, _BOTH, dev)
    if dt_w is None:
        dt_w = FSDP_DTYPE_F32 if dt_b is None else dt_b
    elif dt_b is not None and dt_w != dt_b:
        raise ValueError(f"{where}: weight and bias have different dtypes")
    pm, _, dev = _vector(where, "mean", mean, rows, _F32, dev)
    pr, _, dev = _vector(where, "rstd", rstd, rows, _F32, dev)
    if (mean is None) != (rstd is None):
        raise ValueError(f"{where}: mean and rstd are given together or not at all")
    if rows == 0:
        pm = pr = None
    pk = None
    if keep is not None:
        pk, dev = _ckpt(where, "keep", keep, rows, cols, dev)
    d = fsdp_norm_desc_t(rows, cols, ld_x, ld_y, cols, dt_x, dt_y, FSDP_DTYPE_F32, dt_w, FSDP_DTYPE_F32, eps)
    _check(_lib.fsdp_layer_norm_forward(ctypes.byref(d), px, pw, pb, py, pm, pr, pk, _handle(where, stream, dev)), where)


def fsdp_layer_norm_backward(dy, x, weight, mean, rstd, dx=None, dweight=None, dbias=None, workspace=None,
                             stream=None) -> None:
    """x: a tensor or its ``Act8`` checkpoint; dx, dweight and dbias: what is wanted, written."""
    where = "fsdp_layer_norm_backward"
    py, ld_y, dt_y, dev = _matrix(where, "dy", dy, None, None, _BOTH, None)
    rows, cols = dy.shape
    px, ld_x, dt_x, dev = _norm_input(where, x, rows, cols, dev)
    pw, dt_w, dev = _vector(where, "weight", weight, cols, _BOTH, dev)
    if mean is None or rstd is None:
        raise ValueError(f"{where}: mean and rstd are needed")
    pm, _, dev = _vector(where, "mean", mean, rows, _F32, dev)
    pr, _, dev = _vector(where, "rstd", rstd, rows, _F32, dev)
    pd, ld_d, dt_d = None, cols, FSDP_DTYPE_F32
    if dx is not None:
        pd, ld_d, dt_d, dev = _matrix(where, "dx", dx, rows, cols, _BOTH, dev)
    pdw, dt_dw, dev = _vector(where, "dweight", dweight, cols, _BOTH, dev)
    pdb, dt_db, dev = _vector(where, "dbias", dbias, cols, _BOTH, dev)
    if dt_dw is None:
        dt_dw = FSDP_DTYPE_F32 if dt_db is None else dt_db
    elif dt_db is not None and dt_dw != dt_db:
        raise ValueError(f"{where}: dweight and dbias have different dtypes")
    d = fsdp_norm_desc_t(rows, cols, ld_x, ld_y, ld_d, dt_x, dt_y, dt_d, FSDP_DTYPE_F32 if dt_w is None else dt_w, dt_dw, 0.0)
    handle = _handle(where, stream, dev)
    pws, nws, _owner = _workspace(where, workspace, _norm_workspace(rows, cols, dev), handle, dev)
    _check(_lib.fsdp_layer_norm_backward(ctypes.byref(d), py, px, pw, pm, pr, pd, pdw, pdb, pws, nws, handle), where)


@functools.lru_cache(maxsize=1024)
def _norm_workspace(rows, cols, device) -> int:
    """The size depends on these alone (``device``: its SMs); a program asks for few of them, again and again."""
    d = fsdp_norm_desc_t(rows, cols, cols, cols, cols, 0, 0, 0, 0, 0, 0.0)
    out = _I64()
    _check(_lib.fsdp_layer_norm_workspace(ctypes.byref(d), ctypes.byref(out)), "fsdp_layer_norm_workspace")
    return out.value


def fsdp_layer_norm_workspace(rows: int, cols: int) -> int:
    """Bytes of workspace that fsdp_layer_norm_backward needs for a [rows, cols] matrix."""
    return _norm_workspace(rows, cols, torch.cuda.current_device() if torch.cuda.is_available() else None)


def _kept(where, gate, up, rows, f, dev):
    """(gate pointer, up pointer, row distance, FSDP_KEEP_*, device)."""
    if (gate is None) != (up is None):
        raise ValueError(f"{where}: gate and up are given together or not at all")
    if gate is None:
        return None, None, f, FSDP_KEEP_NONE, dev
    if isinstance(gate, Act8) or isinstance(up, Act8):
        pg, dev = _ckpt(where, "gate", gate, rows, f, dev)
        pu, dev = _ckpt(where, "up", up, rows, f, dev)
        return pg, pu, f, FSDP_KEEP_ACT8, dev
    pg, lg, _, dev = _matrix(where, "gate", gate, rows, f, _BF16, dev)
    pu, lu, _, dev = _matrix(where, "up", up, rows, f, _BF16, dev)
    if lg != lu:
        raise ValueError(f"{where}: gate and up have different row distances")
    return pg, pu, lg, FSDP_KEEP_BF16, dev


@functools.lru_cache(maxsize=1024)
def _ffn_workspace(backward, device, *fields) -> int:
    """By the fields of the descriptor, as for the norm's."""
    d = fsdp_ffn_desc_t(*fields)
    out = _I64()
    _check(_lib.fsdp_gated_ffn_workspace(ctypes.byref(d), backward, ctypes.byref(out)), "fsdp_gated_ffn_workspace")
    return out.value


def fsdp_gated_ffn_workspace(rows: int, d: int, f: int, backward: bool, keep: int = FSDP_KEEP_NONE,
                             x_act8: bool = False, aligned: bool = True) -> int:
    """Bytes of workspace of a call.  ``aligned``: every row of x and of the weights starts on a 16-byte boundary, as those
    of contiguous tensors with d a multiple of 8 do; if not (views at an offset, other row distances), x and both weights
    may have to be copied, and the size is enough for every such call."""
    odd = 0 if aligned and d % 8 == 0 else 7
    return _ffn_workspace(int(backward), torch.cuda.current_device() if torch.cuda.is_available() else None, rows, d, f, d, d, d, f,
                          f, d, d, d, FSDP_ACT_SILU, keep, FSDP_ACT8 if x_act8 else FSDP_DTYPE_BF16, FSDP_DTYPE_BF16,
                          FSDP_DTYPE_BF16, odd)


def fsdp_gated_ffn_forward(x, w_gate, w_up, h, gate=None, up=None, activation=FSDP_ACT_SILU, workspace=None,
                           stream=None) -> None:
    """gate, up: what is kept for the backward pass: ``Act8`` checkpoints, BF16 tensors, or nothing."""
    where = "fsdp_gated_ffn_forward"
    px, ld_x, dt, dev = _matrix(where, "x", x, None, None, _BF16, None)
    rows, d = x.shape
    pg, ld_g, _, dev = _matrix(where, "w_gate", w_gate, None, d, _BF16, dev)
    f = w_gate.shape[0]
    pu, ld_u, _, dev = _matrix(where, "w_up", w_up, f, d, _BF16, dev)
    ph, ld_h, _, dev = _matrix(where, "h", h, rows, f, _BF16, dev)
    pkg, pku, ld_k, keep, dev = _kept(where, gate, up, rows, f, dev)
    off = (px % 16 > 0) + 2 * (pg % 16 > 0) + 4 * (pu % 16 > 0)
    fields = (rows, d, f, ld_x, ld_g, ld_u, ld_h, ld_k, d, d, d, activation, keep, dt, dt, dt, off)
    handle = _handle(where, stream, dev)
    pws, nws, _owner = _workspace(where, workspace, _ffn_workspace(0, dev, *fields), handle, dev)
    _check(_lib.fsdp_gated_ffn_forward(ctypes.byref(fsdp_ffn_desc_t(*fields)), px, pg, pu, ph, pkg, pku, pws, nws, handle), where)


def fsdp_gated_ffn_backward(dh, x, w_gate, w_up, dx=None, dw_gate=None, dw_up=None, gate=None, up=None,
                            activation=FSDP_ACT_SILU, workspace=None, stream=None) -> None:
    """x: the forward pass's input or its ``Act8`` checkpoint; gate, up: as kept (None: computed again);
    dx, dw_gate and dw_up: what is wanted, written."""
    where = "fsdp_gated_ffn_backward"
    pdh, ld_h, dt, dev = _matrix(where, "dh", dh, None, None, _BF16, None)
    rows, f = dh.shape
    pg, ld_g, _, dev = _matrix(where, "w_gate", w_gate, f, None, _BF16, dev)
    d = w_gate.shape[1]
    pu, ld_u, _, dev = _matrix(where, "w_up", w_up, f, d, _BF16, dev)
    off = 2 * (pg % 16 > 0) + 4 * (pu % 16 > 0)
    if isinstance(x, Act8):
        px, dev = _ckpt(where, "x", x, rows, d, dev)
        ld_x, dt_x = d, FSDP_ACT8
    else:
        px, ld_x, dt_x, dev = _matrix(where, "x", x, rows, d, _BF16, dev)
        off += px % 16 > 0
    pkg, pku, ld_k, keep, dev = _kept(where, gate, up, rows, f, dev)
    pdx, ld_dx, dt_dx = None, d, dt
    if dx is not None:
        pdx, ld_dx, dt_dx, dev = _matrix(where, "dx", dx, rows, d, _BOTH, dev)
    if (dw_gate is None) != (dw_up is None):
        raise ValueError(f"{where}: dw_gate and dw_up are given together or not at all")
    pdg = pdu = None
    ld_dg = ld_du = d
    dt_dw = dt
    if dw_gate is not None:
        pdg, ld_dg, dt_dw, dev = _matrix(where, "dw_gate", dw_gate, f, d, _BOTH, dev)
        pdu, ld_du, dt_u, dev = _matrix(where, "dw_up", dw_up, f, d, _BOTH, dev)
        if dt_u != dt_dw:
            raise ValueError(f"{where}: dw_gate and dw_up have different dtypes")
    fields = (rows, d, f, ld_x, ld_g, ld_u, ld_h, ld_k, ld_dx, ld_dg, ld_du, activation, keep, dt_x, dt_dx, dt_dw, off)
    handle = _handle(where, stream, dev)
    pws, nws, _owner = _workspace(where, workspace, _ffn_workspace(1, dev, *fields), handle, dev)
    _check(_lib.fsdp_gated_ffn_backward(ctypes.byref(fsdp_ffn_desc_t(*fields)), pdh, px, pg, pu, pkg, pku, pdx, pdg, pdu, pws, nws,
                                        handle), where)


def fsdp_ops_sync_status(stream=None) -> None:
    """Raises ``FsdpError`` (FSDP_ETIMEOUT) if a wait on this device gave up since this thread last asked."""
    _check(_lib.fsdp_ops_sync_status(_fp._stream(stream)), "fsdp_ops_sync_status")

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
FSDP_INDEX_I32, FSDP_INDEX_I64 = 0, 1
FSDP_DISTILL_MAX_TOP = 1024

__all__ = ["FSDP_ACT8", "FSDP_ACT8_GROUP", "FSDP_NORM_MAX_COLS", "fsdp_norm_desc_t", "Act8", "fsdp_act8_bytes",
           "fsdp_act8_store", "fsdp_act8_load", "fsdp_layer_norm_forward", "fsdp_layer_norm_backward",
           "fsdp_layer_norm_workspace", "FSDP_ACT_SILU", "FSDP_ACT_GELU", "FSDP_KEEP_NONE", "FSDP_KEEP_ACT8",
           "FSDP_KEEP_BF16", "fsdp_ffn_desc_t", "fsdp_gated_ffn_forward", "fsdp_gated_ffn_backward",
           "fsdp_gated_ffn_workspace", "fsdp_ops_sync_status", "FSDP_INDEX_I32", "FSDP_INDEX_I64", "FSDP_DISTILL_MAX_TOP",
           "fsdp_embedding_desc_t", "fsdp_embedding_forward", "fsdp_embedding_backward", "fsdp_embedding_workspace",
           "fsdp_scan_desc_t", "fsdp_gated_scan_forward", "fsdp_gated_scan_backward", "fsdp_gated_scan_states",
           "fsdp_gated_scan_workspace", "fsdp_distill_desc_t", "fsdp_distill_loss_forward", "fsdp_distill_loss_backward",
           "fsdp_policy_desc_t", "fsdp_policy_loss_forward", "fsdp_policy_loss_backward"]

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


class fsdp_embedding_desc_t(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("rows", "vocab", "cols", "ld_weight", "ld_out")] + \
               [(n, ctypes.c_int32) for n in ("token_dtype", "weight_dtype", "out_dtype", "accumulate")] + [("scale", ctypes.c_float)]


class fsdp_scan_desc_t(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("rows", "cols", "seqs", "seq_len", "ld_x", "ld_gate", "ld_h", "ld_dx", "ld_dgate")] + \
               [(n, ctypes.c_int32) for n in ("packed", "offset_dtype", "x_dtype", "h_dtype", "dx_dtype", "param_dtype", "grad_dtype")]


class fsdp_distill_desc_t(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("rows", "vocab", "ld_logits", "ld_dlogits", "top", "ld_tokens", "ld_teacher")] + \
               [(n, ctypes.c_int32) for n in ("logits_dtype", "dlogits_dtype", "teacher_dtype", "token_dtype")] + \
               [("temperature", ctypes.c_float)]


class fsdp_policy_desc_t(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("rows", "vocab", "ld_logits", "ld_dlogits")] + \
               [(n, ctypes.c_int32) for n in ("logits_dtype", "dlogits_dtype", "token_dtype")] + \
               [(n, ctypes.c_float) for n in ("temperature", "clip_low", "clip_high", "kl")]


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
    "fsdp_embedding_forward": [ctypes.POINTER(fsdp_embedding_desc_t)] + [_P] * 4,
    "fsdp_embedding_backward": [ctypes.POINTER(fsdp_embedding_desc_t)] + [_P] * 4 + [_I64, _P],
    "fsdp_embedding_workspace": [ctypes.POINTER(fsdp_embedding_desc_t), ctypes.POINTER(_I64)],
    "fsdp_gated_scan_states": [_I64, _I64, ctypes.POINTER(_I64)],
    "fsdp_gated_scan_workspace": [ctypes.POINTER(fsdp_scan_desc_t), _I32, ctypes.POINTER(_I64)],
    "fsdp_gated_scan_forward": [ctypes.POINTER(fsdp_scan_desc_t)] + [_P] * 9 + [_I64, _P],
    "fsdp_gated_scan_backward": [ctypes.POINTER(fsdp_scan_desc_t)] + [_P] * 13 + [_I64, _P],
    "fsdp_distill_loss_forward": [ctypes.POINTER(fsdp_distill_desc_t)] + [_P] * 8,
    "fsdp_distill_loss_backward": [ctypes.POINTER(fsdp_distill_desc_t)] + [_P] * 8,
    "fsdp_policy_loss_forward": [ctypes.POINTER(fsdp_policy_desc_t)] + [_P] * 11,
    "fsdp_policy_loss_backward": [ctypes.POINTER(fsdp_policy_desc_t)] + [_P] * 11,
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
_INDEX = {torch.int32: FSDP_INDEX_I32, torch.int64: FSDP_INDEX_I64}
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


# ---------------------------------------------------------------------------
# Embedding
# ---------------------------------------------------------------------------
def _tokens(where, what, t, device):
    """(pointer, count, dtype code, device) of a contiguous tensor of token ids, of any shape."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{where}: {what} is not a tensor")
    code = _INDEX.get(t.dtype)
    if code is None:
        raise ValueError(f"{where}: {what} is {t.dtype}, not one of {', '.join(map(str, _INDEX))}")
    if not t.is_contiguous():
        raise ValueError(f"{where}: {what} is not contiguous")
    index = t.get_device()
    if index != device:
        _misplaced(where, what, index, device)
    return t.data_ptr(), t.numel(), code, index


def fsdp_embedding_forward(tokens, weight, out, scale=1.0, stream=None) -> None:
    """out[i] = scale * weight[tokens[i]]; tokens of any shape, those outside the vocabulary give rows of zeros."""
    where = "fsdp_embedding_forward"
    pt, rows, dt_t, dev = _tokens(where, "tokens", tokens, None)
    pw, ld_w, dt_w, dev = _matrix(where, "weight", weight, None, None, _BOTH, dev)
    vocab, cols = weight.shape
    po, ld_o, dt_o, dev = _matrix(where, "out", out, rows, cols, _BOTH, dev)
    d = fsdp_embedding_desc_t(rows, vocab, cols, ld_w, ld_o, dt_t, dt_w, dt_o, 0, scale)
    _check(_lib.fsdp_embedding_forward(ctypes.byref(d), pt, pw, po, _handle(where, stream, dev)), where)


@functools.lru_cache(maxsize=1024)
def _embedding_workspace(rows, vocab, cols) -> int:
    d = fsdp_embedding_desc_t(rows, vocab, cols, cols, cols, 0, 0, 0, 0, 1.0)
    out = _I64()
    _check(_lib.fsdp_embedding_workspace(ctypes.byref(d), ctypes.byref(out)), "fsdp_embedding_workspace")
    return out.value


def fsdp_embedding_workspace(rows: int, vocab: int, cols: int) -> int:
    """Bytes of workspace that fsdp_embedding_backward needs for that many tokens and a [vocab, cols] gradient."""
    return _embedding_workspace(rows, vocab, cols)


def fsdp_embedding_backward(tokens, dout, dweight, scale=1.0, accumulate=False, workspace=None, stream=None) -> None:
    """dweight[v] = scale * sum of dout's rows of token v, written whole, or added where ``accumulate``."""
    where = "fsdp_embedding_backward"
    pt, rows, dt_t, dev = _tokens(where, "tokens", tokens, None)
    pw, ld_w, dt_w, dev = _matrix(where, "dweight", dweight, None, None, _BOTH, dev)
    vocab, cols = dweight.shape
    po, ld_o, dt_o, dev = _matrix(where, "dout", dout, rows, cols, _BOTH, dev)
    d = fsdp_embedding_desc_t(rows, vocab, cols, ld_w, ld_o, dt_t, dt_w, dt_o, bool(accumulate), scale)
    handle = _handle(where, stream, dev)
    pws, nws, _owner = _workspace(where, workspace, _embedding_workspace(rows, vocab, cols), handle, dev)
    _check(_lib.fsdp_embedding_backward(ctypes.byref(d), pt, po, pw, pws, nws, handle), where)


# ---------------------------------------------------------------------------
# Gated linear recurrence
# ---------------------------------------------------------------------------
def fsdp_gated_scan_states(rows: int, cols: int) -> int:
    """Rows of the FP32 matrix [n, cols] that a forward call fills for the backward call."""
    out = _I64()
    _check(_lib.fsdp_gated_scan_states(rows, cols, ctypes.byref(out)), "fsdp_gated_scan_states")
    return out.value


@functools.lru_cache(maxsize=1024)
def _scan_workspace(rows, cols, seqs, packed, backward) -> int:
    d = fsdp_scan_desc_t(rows, cols, seqs, 1 if packed or not seqs else rows // seqs, cols, cols, cols, cols, cols, packed, 0, 0, 0, 0, 0, 0)
    out = _I64()
    _check(_lib.fsdp_gated_scan_workspace(ctypes.byref(d), backward, ctypes.byref(out)), "fsdp_gated_scan_workspace")
    return out.value


def fsdp_gated_scan_workspace(rows: int, cols: int, seqs: int, packed: bool, backward: bool) -> int:
    """Bytes of workspace of a call over ``seqs`` sequences in ``rows`` rows."""
    return _scan_workspace(rows, cols, seqs, int(packed), int(backward))


def _sequences(where, rows, seq_len, offsets, dev):
    """(sequences, rows of each, offsets pointer, their dtype code, device)."""
    if (seq_len is None) == (offsets is None):
        raise ValueError(f"{where}: either seq_len or offsets is needed")
    if offsets is None:
        if seq_len < 1 or rows % seq_len:
            raise ValueError(f"{where}: {rows} rows are not sequences of {seq_len}")
        return rows // seq_len, seq_len, None, 0, dev
    po, n, code, dev = _tokens(where, "offsets", offsets, dev)
    if n < 1:
        raise ValueError(f"{where}: offsets is empty")
    return n - 1, 0, po, code, dev


def _states(where, what, t, rows, cols, dev):
    """(pointer, device) of a contiguous FP32 matrix [rows, cols], or of nothing."""
    if t is None:
        return None, dev
    p, ld, _, dev = _matrix(where, what, t, rows, cols, _F32, dev)
    if ld != cols:
        raise ValueError(f"{where}: {what} has gaps between its rows")
    return p, dev


def fsdp_gated_scan_forward(x, gate, h, bias=None, initial=None, final=None, seq_len=None, offsets=None, states=None,
                            workspace=None, stream=None) -> None:
    """Sequences of ``seq_len`` rows each, or from ``offsets[s]`` up to ``offsets[s + 1]``.  initial, final: FP32
    [sequences, cols] (may be one tensor); states: FP32 [fsdp_gated_scan_states(rows, cols), cols] for the backward pass."""
    where = "fsdp_gated_scan_forward"
    px, ld_x, dt_x, dev = _matrix(where, "x", x, None, None, _BOTH, None)
    rows, cols = x.shape
    pg, ld_g, dt_g, dev = _matrix(where, "gate", gate, rows, cols, _BOTH, dev)
    if dt_g != dt_x:
        raise ValueError(f"{where}: x and gate have different dtypes")
    ph, ld_h, dt_h, dev = _matrix(where, "h", h, rows, cols, _BOTH, dev)
    pb, dt_b, dev = _vector(where, "bias", bias, cols, _BOTH, dev)
    seqs, length, po, dt_o, dev = _sequences(where, rows, seq_len, offsets, dev)
    pi, dev = _states(where, "initial", initial, seqs, cols, dev)
    pf, dev = _states(where, "final", final, seqs, cols, dev)
    ps = None
    if states is not None:
        ps, dev = _states(where, "states", states, fsdp_gated_scan_states(rows, cols), cols, dev)
    packed = po is not None
    d = fsdp_scan_desc_t(rows, cols, seqs, length, ld_x, ld_g, ld_h, cols, cols, packed, dt_o, dt_x, dt_h, FSDP_DTYPE_F32,
                         FSDP_DTYPE_F32 if dt_b is None else dt_b, FSDP_DTYPE_F32)
    handle = _handle(where, stream, dev)
    pws, nws, _owner = _workspace(where, workspace, _scan_workspace(rows, cols, seqs, int(packed), 0), handle, dev)
    _check(_lib.fsdp_gated_scan_forward(ctypes.byref(d), px, pg, pb, pi, po, ph, pf, ps, pws, nws, handle), where)


def fsdp_gated_scan_backward(dh, x, gate, states, dx, dgate, bias=None, dbias=None, initial=None, dinitial=None, dfinal=None,
                             seq_len=None, offsets=None, workspace=None, stream=None) -> None:
    """states: as the forward call wrote them; dbias and dinitial: written if given."""
    where = "fsdp_gated_scan_backward"
    ph, ld_h, dt_h, dev = _matrix(where, "dh", dh, None, None, _BOTH, None)
    rows, cols = dh.shape
    px, ld_x, dt_x, dev = _matrix(where, "x", x, rows, cols, _BOTH, dev)
    pg, ld_g, dt_g, dev = _matrix(where, "gate", gate, rows, cols, _BOTH, dev)
    if dt_g != dt_x:
        raise ValueError(f"{where}: x and gate have different dtypes")
    pdx, ld_dx, dt_dx, dev = _matrix(where, "dx", dx, rows, cols, _BOTH, dev)
    pdg, ld_dg, dt_dg, dev = _matrix(where, "dgate", dgate, rows, cols, _BOTH, dev)
    if dt_dg != dt_dx:
        raise ValueError(f"{where}: dx and dgate have different dtypes")
    pb, dt_b, dev = _vector(where, "bias", bias, cols, _BOTH, dev)
    pdb, dt_db, dev = _vector(where, "dbias", dbias, cols, _BOTH, dev)
    seqs, length, po, dt_o, dev = _sequences(where, rows, seq_len, offsets, dev)
    if states is None:
        raise ValueError(f"{where}: states is needed")
    ps, dev = _states(where, "states", states, fsdp_gated_scan_states(rows, cols), cols, dev)
    pi, dev = _states(where, "initial", initial, seqs, cols, dev)
    pdi, dev = _states(where, "dinitial", dinitial, seqs, cols, dev)
    pdf, dev = _states(where, "dfinal", dfinal, seqs, cols, dev)
    packed = po is not None
    d = fsdp_scan_desc_t(rows, cols, seqs, length, ld_x, ld_g, ld_h, ld_dx, ld_dg, packed, dt_o, dt_x, dt_h, dt_dx,
                         FSDP_DTYPE_F32 if dt_b is None else dt_b, FSDP_DTYPE_F32 if dt_db is None else dt_db)
    handle = _handle(where, stream, dev)
    pws, nws, _owner = _workspace(where, workspace, _scan_workspace(rows, cols, seqs, int(packed), 1), handle, dev)
    _check(_lib.fsdp_gated_scan_backward(ctypes.byref(d), ph, px, pg, pb, pi, po, ps, pdf, pdx, pdg, pdb, pdi, pws, nws, handle), where)


# ---------------------------------------------------------------------------
# Losses over logits
# ---------------------------------------------------------------------------
def _entries(where, what, t, rows, top, codes, device):
    """As _matrix, of a teacher's entries: a row may have none."""
    if not isinstance(t, torch.Tensor) or t.dim() != 2 or t.shape[1] > 0 or top:
        return _matrix(where, what, t, rows, top, codes, device)
    if t.shape[0] != rows:
        raise ValueError(f"{where}: {what} is {t.shape[0]} x 0, not {rows} x 0")
    code = codes.get(t.dtype)
    if code is None:
        raise ValueError(f"{where}: {what} is {t.dtype}, not one of {', '.join(map(str, codes))}")
    if t.get_device() != device:
        _misplaced(where, what, t.get_device(), device)
    return None, 0, code, device


def _distill(where, logits, dlogits, teacher_tokens, teacher_logits, weight, temperature):
    """(descriptor, pointers of logits, dlogits, tokens, teacher and weight, device)."""
    pz, ld_z, dt_z, dev = _matrix(where, "logits", logits, None, None, _BOTH, None)
    rows, vocab = logits.shape
    pd, ld_d, dt_d = None, vocab, dt_z
    if dlogits is not None:
        pd, ld_d, dt_d, dev = _matrix(where, "dlogits", dlogits, rows, vocab, _BOTH, dev)
    pi, ld_i, dt_i, dev = _entries(where, "teacher_tokens", teacher_tokens, rows, None, _INDEX, dev)
    top = teacher_tokens.shape[1]
    pt, ld_t, dt_t, dev = _entries(where, "teacher_logits", teacher_logits, rows, top, _BOTH, dev)
    pw, _, dev = _vector(where, "weight", weight, rows, _F32, dev)
    return fsdp_distill_desc_t(rows, vocab, ld_z, ld_d, top, ld_i, ld_t, dt_z, dt_d, dt_t, dt_i, temperature), pz, pd, pi, pt, pw, dev


def _needed(where, what, t, n, codes, dev):
    if t is None:
        raise ValueError(f"{where}: {what} is needed")
    p, _, dev = _vector(where, what, t, n, codes, dev)
    return p, dev


def fsdp_distill_loss_forward(logits, teacher_tokens, teacher_logits, loss, lse, temperature=1.0, weight=None, dlogits=None,
                              stream=None) -> None:
    """Rows' losses against a teacher's top logits [rows, top]; dlogits: receives the gradient of their sum in the same
    pass (it may be ``logits`` itself)."""
    where = "fsdp_distill_loss_forward"
    d, pz, pd, pi, pt, pw, dev = _distill(where, logits, dlogits, teacher_tokens, teacher_logits, weight, temperature)
    pl, dev = _needed(where, "loss", loss, d.rows, _F32, dev)
    pe, dev = _needed(where, "lse", lse, d.rows, _F32, dev)
    _check(_lib.fsdp_distill_loss_forward(ctypes.byref(d), pz, pi, pt, pw, pl, pe, pd, _handle(where, stream, dev)), where)


def fsdp_distill_loss_backward(logits, teacher_tokens, teacher_logits, lse, dlogits, temperature=1.0, weight=None, dloss=None,
                               stream=None) -> None:
    """dlogits from the lse of a forward call; dloss: the gradient of each row's loss (None: 1)."""
    where = "fsdp_distill_loss_backward"
    if dlogits is None:
        raise ValueError(f"{where}: dlogits is needed")
    d, pz, pd, pi, pt, pw, dev = _distill(where, logits, dlogits, teacher_tokens, teacher_logits, weight, temperature)
    pe, dev = _needed(where, "lse", lse, d.rows, _F32, dev)
    pu, _, dev = _vector(where, "dloss", dloss, d.rows, _F32, dev)
    _check(_lib.fsdp_distill_loss_backward(ctypes.byref(d), pz, pi, pt, pw, pe, pu, pd, _handle(where, stream, dev)), where)


def _policy(where, logits, dlogits, tokens, old_logp, ref_logp, advantage, weight, temperature, clip_low, clip_high, kl):
    """(descriptor, pointers of logits, dlogits, tokens, old_logp, ref_logp, advantage and weight, device)."""
    pz, ld_z, dt_z, dev = _matrix(where, "logits", logits, None, None, _BOTH, None)
    rows, vocab = logits.shape
    pd, ld_d, dt_d = None, vocab, dt_z
    if dlogits is not None:
        pd, ld_d, dt_d, dev = _matrix(where, "dlogits", dlogits, rows, vocab, _BOTH, dev)
    pi, n, dt_i, dev = _tokens(where, "tokens", tokens, dev)
    if n != rows:
        raise ValueError(f"{where}: {n} tokens for {rows} rows")
    po, _, dev = _vector(where, "old_logp", old_logp, rows, _F32, dev)
    pr, _, dev = _vector(where, "ref_logp", ref_logp, rows, _F32, dev)
    pa, dev = _needed(where, "advantage", advantage, rows, _F32, dev)
    pw, _, dev = _vector(where, "weight", weight, rows, _F32, dev)
    d = fsdp_policy_desc_t(rows, vocab, ld_z, ld_d, dt_z, dt_d, dt_i, temperature, clip_low, clip_high, kl)
    return d, pz, pd, pi, po, pr, pa, pw, dev


def fsdp_policy_loss_forward(logits, tokens, old_logp, advantage, loss, logp, lse, ref_logp=None, weight=None, temperature=1.0,
                             clip_low=0.2, clip_high=0.2, kl=0.0, dlogits=None, stream=None) -> None:
    """Rows' losses and the log-probabilities of their tokens; old_logp None: the policy itself; dlogits: receives the
    gradient of the losses' sum in the same pass (it may be ``logits`` itself)."""
    where = "fsdp_policy_loss_forward"
    d, pz, pd, pi, po, pr, pa, pw, dev = _policy(where, logits, dlogits, tokens, old_logp, ref_logp, advantage, weight, temperature,
                                                 clip_low, clip_high, kl)
    pl, dev = _needed(where, "loss", loss, d.rows, _F32, dev)
    pp, dev = _needed(where, "logp", logp, d.rows, _F32, dev)
    pe, dev = _needed(where, "lse", lse, d.rows, _F32, dev)
    _check(_lib.fsdp_policy_loss_forward(ctypes.byref(d), pz, pi, po, pr, pa, pw, pl, pp, pe, pd, _handle(where, stream, dev)), where)


def fsdp_policy_loss_backward(logits, tokens, old_logp, advantage, logp, lse, dlogits, ref_logp=None, weight=None, dloss=None,
                              temperature=1.0, clip_low=0.2, clip_high=0.2, kl=0.0, stream=None) -> None:
    """dlogits from the logp and lse of a forward call; dloss: the gradient of each row's loss (None: 1)."""
    where = "fsdp_policy_loss_backward"
    if dlogits is None:
        raise ValueError(f"{where}: dlogits is needed")
    d, pz, pd, pi, po, pr, pa, pw, dev = _policy(where, logits, dlogits, tokens, old_logp, ref_logp, advantage, weight, temperature,
                                                 clip_low, clip_high, kl)
    pp, dev = _needed(where, "logp", logp, d.rows, _F32, dev)
    pe, dev = _needed(where, "lse", lse, d.rows, _F32, dev)
    pu, _, dev = _vector(where, "dloss", dloss, d.rows, _F32, dev)
    _check(_lib.fsdp_policy_loss_backward(ctypes.byref(d), pz, pi, po, pr, pa, pw, pp, pe, pu, pd, _handle(where, stream, dev)), where)


def fsdp_ops_sync_status(stream=None) -> None:
    """Raises ``FsdpError`` (FSDP_ETIMEOUT) if a wait on this device gave up since this thread last asked."""
    _check(_lib.fsdp_ops_sync_status(_fp._stream(stream)), "fsdp_ops_sync_status")

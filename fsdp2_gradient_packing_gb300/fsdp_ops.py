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
# Arguments
# ---------------------------------------------------------------------------
class _Args:
    """Checks the tensors of one call: where they are, and their shapes and dtypes."""

    def __init__(self, where):
        self.where, self.device = where, None

    def fail(self, why):
        raise ValueError(f"{self.where}: {why}")

    def _placed(self, what, t):
        if not isinstance(t, torch.Tensor):
            self.fail(f"{what} is not a tensor")
        index = t.get_device()
        if index < 0:
            self.fail(f"{what} is not a CUDA tensor")
        if self.device is None:
            self.device = index
        elif index != self.device:
            self.fail(f"{what} is on cuda:{index}, another argument on cuda:{self.device}")

    def matrix(self, what, t, rows=None, cols=None, dtypes=(torch.float32, torch.bfloat16)):
        """(pointer, row distance, dtype code) of a [rows, cols] tensor."""
        if not isinstance(t, torch.Tensor):
            self.fail(f"{what} is not a tensor")
        if t.dim() != 2:
            self.fail(f"{what} has {t.dim()} dimensions, not 2")
        r, c = t.shape
        if (rows is not None and r != rows) or (cols is not None and c != cols):
            self.fail(f"{what} is {r} x {c}, not {r if rows is None else rows} x {c if cols is None else cols}")
        if t.dtype not in dtypes:
            self.fail(f"{what} is {t.dtype}, not one of {', '.join(map(str, dtypes))}")
        if c < 1:
            self.fail(f"{what} has no columns")
        s0, s1 = t.stride()
        if c > 1 and s1 != 1:
            self.fail(f"{what} has column stride {s1}, not 1")
        if r <= 1:
            s0 = c
        elif s0 < c:
            self.fail(f"{what} has rows {s0} elements apart, fewer than its {c} columns")
        self._placed(what, t)
        return t.data_ptr(), s0, _CODE[t.dtype]

    def vector(self, what, t, n, dtypes=(torch.float32, torch.bfloat16)):
        """(pointer, dtype code) of a contiguous vector of n elements; (None, None) for None."""
        if t is None:
            return None, None
        if not isinstance(t, torch.Tensor):
            self.fail(f"{what} is not a tensor")
        if t.numel() != n or t.dim() > 1 and t.shape[-1] != n or not t.is_contiguous():
            self.fail(f"{what} is not a contiguous vector of {n} elements")
        if t.dtype not in dtypes:
            self.fail(f"{what} is {t.dtype}, not one of {', '.join(map(str, dtypes))}")
        self._placed(what, t)
        return t.data_ptr(), _CODE[t.dtype]

    def ckpt(self, what, a, rows=None, cols=None):
        if not isinstance(a, Act8):
            self.fail(f"{what} is not an Act8 checkpoint")
        if (rows is not None and a.rows != rows) or (cols is not None and a.cols != cols):
            self.fail(f"{what} is a checkpoint of {a.rows} x {a.cols}, not of {rows} x {cols}")
        self._placed(what, a.data)
        return a.data.data_ptr()

    def stream(self, stream):
        """The handle of the stream to run on; the tensors have to be on the current device."""
        if self.device is not None and self.device != torch.cuda.current_device():
            self.fail(f"the tensors are on cuda:{self.device}, the current device is {torch.cuda.current_device()}")
        if stream is None:
            return _current_stream()
        return stream if isinstance(stream, int) else stream.cuda_stream

    def workspace(self, given, nbytes, handle):
        """(pointer, bytes, owner) of the caller's workspace or of one taken for this call."""
        if given is not None:
            if given.dtype != torch.uint8 or not given.is_contiguous():
                self.fail("workspace is not a contiguous uint8 tensor")
            self._placed("workspace", given)
            if given.numel() < nbytes:
                self.fail(f"workspace holds {given.numel()} bytes, the call needs {nbytes}")
            return given.data_ptr(), given.numel(), given
        ws = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=f"cuda:{self.device}")
        if handle != _current_stream():  # the allocator may not reuse it before the call's stream is done with it
            ws.record_stream(torch.cuda.ExternalStream(handle) if handle else torch.cuda.default_stream())
        return ws.data_ptr(), nbytes, ws


class Act8:
    """The 8-bit checkpoint of a ``[rows, cols]`` matrix: one uint8 tensor, codes ``[rows, 32 G]`` and then scale
    bytes ``[rows, G]`` with ``G = ceil(cols / 32)``.  ``data``: a buffer to use instead of a new one."""

    __slots__ = ("rows", "cols", "data")

    def __init__(self, rows, cols, data=None, device="cuda"):
        nbytes = fsdp_act8_bytes(rows, cols)
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
    a = _Args("fsdp_act8_store")
    p, ld, dt = a.matrix("x", x)
    c = a.ckpt("ckpt", ckpt, x.shape[0], x.shape[1])
    _check(_lib.fsdp_act8_store(p, dt, ckpt.rows, ckpt.cols, ld, c, a.stream(stream)), "fsdp_act8_store")


def fsdp_act8_load(ckpt: Act8, y, stream=None) -> None:
    a = _Args("fsdp_act8_load")
    p, ld, dt = a.matrix("y", y)
    c = a.ckpt("ckpt", ckpt, y.shape[0], y.shape[1])
    _check(_lib.fsdp_act8_load(c, ckpt.rows, ckpt.cols, p, dt, ld, a.stream(stream)), "fsdp_act8_load")


def _norm_input(a: _Args, x, rows, cols):
    """(pointer, row distance, dtype code) of a norm's input, a tensor or a checkpoint."""
    if isinstance(x, Act8):
        return a.ckpt("x", x, rows, cols), cols, FSDP_ACT8
    return a.matrix("x", x, rows, cols)


def fsdp_layer_norm_forward(x, weight, bias, y, mean=None, rstd=None, eps=1e-5, keep=None, stream=None) -> None:
    """x: a tensor or its ``Act8`` checkpoint; keep: an ``Act8`` that receives x's checkpoint in the same pass."""
    a = _Args("fsdp_layer_norm_forward")
    py, ld_y, dt_y = a.matrix("y", y)
    rows, cols = y.shape
    px, ld_x, dt_x = _norm_input(a, x, rows, cols)
    pw, dt_w = a.vector("weight", weight, cols)
    pb, dt_b = a.vector("bias", bias, cols)
    if dt_w is not None and dt_b is not None and dt_w != dt_b:
        a.fail("weight and bias have different dtypes")
    f32 = (torch.float32,)
    pm, pr = a.vector("mean", mean, rows, f32)[0], a.vector("rstd", rstd, rows, f32)[0]
    pk = None if keep is None else a.ckpt("keep", keep, rows, cols)
    d = fsdp_norm_desc_t(rows, cols, ld_x, ld_y, cols, dt_x, dt_y, FSDP_DTYPE_F32,
                         dt_w if dt_w is not None else dt_b if dt_b is not None else FSDP_DTYPE_F32, FSDP_DTYPE_F32, eps)
    if rows and (pm is None) != (pr is None):
        a.fail("mean and rstd are given together or not at all")
    if rows == 0:
        pm = pr = None
    _check(_lib.fsdp_layer_norm_forward(ctypes.byref(d), px, pw, pb, py, pm, pr, pk, a.stream(stream)),
           "fsdp_layer_norm_forward")


def fsdp_layer_norm_backward(dy, x, weight, mean, rstd, dx=None, dweight=None, dbias=None, workspace=None,
                             stream=None) -> None:
    """x: a tensor or its ``Act8`` checkpoint; dx, dweight and dbias: what is wanted, written."""
    a = _Args("fsdp_layer_norm_backward")
    py, ld_y, dt_y = a.matrix("dy", dy)
    rows, cols = dy.shape
    px, ld_x, dt_x = _norm_input(a, x, rows, cols)
    pw, dt_w = a.vector("weight", weight, cols)
    f32 = (torch.float32,)
    if mean is None or rstd is None:
        a.fail("mean and rstd are needed")
    pm, pr = a.vector("mean", mean, rows, f32)[0], a.vector("rstd", rstd, rows, f32)[0]
    pd, ld_d, dt_d = (None, cols, FSDP_DTYPE_F32) if dx is None else a.matrix("dx", dx, rows, cols)
    pdw, dt_dw = a.vector("dweight", dweight, cols)
    pdb, dt_db = a.vector("dbias", dbias, cols)
    if dt_dw is not None and dt_db is not None and dt_dw != dt_db:
        a.fail("dweight and dbias have different dtypes")
    d = fsdp_norm_desc_t(rows, cols, ld_x, ld_y, ld_d, dt_x, dt_y, dt_d, dt_w if dt_w is not None else FSDP_DTYPE_F32,
                         dt_dw if dt_dw is not None else dt_db if dt_db is not None else FSDP_DTYPE_F32, 0.0)
    handle = a.stream(stream)
    pws, nws, _owner = a.workspace(workspace, _norm_workspace(d), handle)
    _check(_lib.fsdp_layer_norm_backward(ctypes.byref(d), py, px, pw, pm, pr, pd, pdw, pdb, pws, nws, handle),
           "fsdp_layer_norm_backward")


def _norm_workspace(d) -> int:
    out = _I64()
    _check(_lib.fsdp_layer_norm_workspace(ctypes.byref(d), ctypes.byref(out)), "fsdp_layer_norm_workspace")
    return out.value


def fsdp_layer_norm_workspace(rows: int, cols: int) -> int:
    """Bytes of workspace that fsdp_layer_norm_backward needs for a [rows, cols] matrix."""
    return _norm_workspace(fsdp_norm_desc_t(rows, cols, cols, cols, cols, 0, 0, 0, 0, 0, 0.0))


_BF16_ONLY = (torch.bfloat16,)


def _kept(a: _Args, gate, up, rows, f):
    """(gate pointer, up pointer, row distance, FSDP_KEEP_*)."""
    if (gate is None) != (up is None):
        a.fail("gate and up are given together or not at all")
    if gate is None:
        return None, None, f, FSDP_KEEP_NONE
    if isinstance(gate, Act8) or isinstance(up, Act8):
        return a.ckpt("gate", gate, rows, f), a.ckpt("up", up, rows, f), f, FSDP_KEEP_ACT8
    pg, lg, _ = a.matrix("gate", gate, rows, f, _BF16_ONLY)
    pu, lu, _ = a.matrix("up", up, rows, f, _BF16_ONLY)
    if lg != lu:
        a.fail("gate and up have different row distances")
    return pg, pu, lg, FSDP_KEEP_BF16


def _ffn_workspace(d, backward) -> int:
    out = _I64()
    _check(_lib.fsdp_gated_ffn_workspace(ctypes.byref(d), backward, ctypes.byref(out)), "fsdp_gated_ffn_workspace")
    return out.value


def fsdp_gated_ffn_workspace(rows: int, d: int, f: int, backward: bool, keep: int = FSDP_KEEP_NONE,
                             x_act8: bool = False) -> int:
    """Bytes of workspace of a call on contiguous matrices, d and f multiples of 8, that start on 16-byte boundaries;
    for others, an upper bound with everything that may have to be copied."""
    odd = 0 if d % 8 == 0 else 7
    desc = fsdp_ffn_desc_t(rows, d, f, d, d, d, f, f, d, d, d, FSDP_ACT_SILU, keep,
                           FSDP_ACT8 if x_act8 else FSDP_DTYPE_BF16, FSDP_DTYPE_BF16, FSDP_DTYPE_BF16, odd)
    return _ffn_workspace(desc, int(backward))


def _off16(*ptrs) -> int:
    return sum(1 << i for i, p in enumerate(ptrs) if p is not None and p % 16)


def fsdp_gated_ffn_forward(x, w_gate, w_up, h, gate=None, up=None, activation=FSDP_ACT_SILU, workspace=None,
                           stream=None) -> None:
    """gate, up: what is kept for the backward pass: ``Act8`` checkpoints, BF16 tensors, or nothing."""
    a = _Args("fsdp_gated_ffn_forward")
    px, ld_x, _ = a.matrix("x", x, dtypes=_BF16_ONLY)
    rows, d = x.shape
    pg, ld_g, _ = a.matrix("w_gate", w_gate, None, d, _BF16_ONLY)
    f = w_gate.shape[0]
    pu, ld_u, _ = a.matrix("w_up", w_up, f, d, _BF16_ONLY)
    ph, ld_h, _ = a.matrix("h", h, rows, f, _BF16_ONLY)
    pkg, pku, ld_k, keep = _kept(a, gate, up, rows, f)
    desc = fsdp_ffn_desc_t(rows, d, f, ld_x, ld_g, ld_u, ld_h, ld_k, d, d, d, activation, keep, FSDP_DTYPE_BF16,
                           FSDP_DTYPE_BF16, FSDP_DTYPE_BF16, _off16(px, pg, pu))
    handle = a.stream(stream)
    pws, nws, _owner = a.workspace(workspace, _ffn_workspace(desc, 0), handle)
    _check(_lib.fsdp_gated_ffn_forward(ctypes.byref(desc), px, pg, pu, ph, pkg, pku, pws, nws, handle),
           "fsdp_gated_ffn_forward")


def fsdp_gated_ffn_backward(dh, x, w_gate, w_up, dx=None, dw_gate=None, dw_up=None, gate=None, up=None,
                            activation=FSDP_ACT_SILU, workspace=None, stream=None) -> None:
    """x: the forward pass's input or its ``Act8`` checkpoint; gate, up: as kept (None: computed again);
    dx, dw_gate and dw_up: what is wanted, written."""
    a = _Args("fsdp_gated_ffn_backward")
    pdh, ld_h, _ = a.matrix("dh", dh, dtypes=_BF16_ONLY)
    rows, f = dh.shape
    pg, ld_g, _ = a.matrix("w_gate", w_gate, f, None, _BF16_ONLY)
    d = w_gate.shape[1]
    pu, ld_u, _ = a.matrix("w_up", w_up, f, d, _BF16_ONLY)
    if isinstance(x, Act8):
        px, ld_x, dt_x = a.ckpt("x", x, rows, d), d, FSDP_ACT8
    else:
        px, ld_x, dt_x = a.matrix("x", x, rows, d, _BF16_ONLY)
    pkg, pku, ld_k, keep = _kept(a, gate, up, rows, f)
    pdx, ld_dx, dt_dx = (None, d, FSDP_DTYPE_BF16) if dx is None else a.matrix("dx", dx, rows, d)
    if (dw_gate is None) != (dw_up is None):
        a.fail("dw_gate and dw_up are given together or not at all")
    pdg = pdu = None
    ld_dg = ld_du = d
    dt_dw = FSDP_DTYPE_BF16
    if dw_gate is not None:
        pdg, ld_dg, dt_dw = a.matrix("dw_gate", dw_gate, f, d)
        pdu, ld_du, dt_u = a.matrix("dw_up", dw_up, f, d)
        if dt_u != dt_dw:
            a.fail("dw_gate and dw_up have different dtypes")
    desc = fsdp_ffn_desc_t(rows, d, f, ld_x, ld_g, ld_u, ld_h, ld_k, ld_dx, ld_dg, ld_du, activation, keep, dt_x, dt_dx,
                           dt_dw, _off16(None if dt_x == FSDP_ACT8 else px, pg, pu))
    handle = a.stream(stream)
    pws, nws, _owner = a.workspace(workspace, _ffn_workspace(desc, 1), handle)
    _check(_lib.fsdp_gated_ffn_backward(ctypes.byref(desc), pdh, px, pg, pu, pkg, pku, pdx, pdg, pdu, pws, nws, handle),
           "fsdp_gated_ffn_backward")


def fsdp_ops_sync_status(stream=None) -> None:
    a = _Args("fsdp_ops_sync_status")
    _check(_lib.fsdp_ops_sync_status(a.stream(stream)), "fsdp_ops_sync_status")

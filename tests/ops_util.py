"""Plain 64-bit definitions of the training operators, and strided device
matrices between guard bytes, for their GPU tests."""
from __future__ import annotations

import math

import numpy as np
import torch

GUARD = 4096
FILL = 0xA5
F32, BF16, F64 = torch.float32, torch.bfloat16, torch.float64
EPS32 = 2.0 ** -24   # half an ulp of 1 in binary32
HALF = {F32: 2.0 ** -24, BF16: 2.0 ** -8}  # half an ulp of 1: binary32 has 24 significant bits, BF16 has 8


class Matrix:
    """A [rows, cols] device matrix whose rows are ``ld`` elements apart, starting ``offset`` elements past a 512-byte
    boundary, with guard bytes before, after and between the rows."""

    def __init__(self, rows, cols, dtype, ld=None, offset=0, value=None):
        self.rows, self.cols, self.ld = rows, cols, cols if ld is None else ld
        size = torch.empty(0, dtype=dtype).element_size()
        self.span = ((max(rows, 1) - 1) * self.ld + cols) * size if rows else 0
        self.start = GUARD + offset * size
        self.raw = torch.full((self.start + max(rows, 1) * self.ld * size + GUARD,), FILL, dtype=torch.uint8, device="cuda")
        flat = self.raw[self.start:self.start + max(rows, 1) * self.ld * size].view(dtype)
        self.t = flat.view(max(rows, 1), self.ld)[:rows, :cols]
        if value is not None:
            self.t.copy_(value)

    def intact(self):
        """Whether everything outside the matrix still holds the guard value."""
        keep = self.t.clone()
        self.t.view(torch.int16 if self.t.dtype == BF16 else torch.int32).fill_(-0x5A5B if self.t.dtype == BF16 else -0x5A5A5A5B)
        ok = bool((self.raw == FILL).all().item())
        self.t.copy_(keep)
        return ok


def act8_encode(x):
    """(codes [rows, 32 G] int8, scale bytes [rows, G] uint8) of a float64 CPU matrix, from the definition."""
    x = np.asarray(x, dtype=np.float64)
    rows, cols = x.shape
    groups = (cols + 31) // 32
    pad = np.zeros((rows, groups * 32))
    pad[:, :cols] = x
    pad = pad.reshape(rows, groups, 32)
    top = np.abs(pad).max(-1)  # NaN where the group holds one
    fine = np.isfinite(top)
    part, e = np.frexp(np.where(fine, top, 1.0) / 127)
    e = np.maximum(np.where(part == 0.5, e - 1, e), -126)
    e = np.where(top == 0, -126, e)
    codes = np.rint(np.ldexp(np.where(fine[..., None], pad, 0.0), -e[..., None]))
    codes = np.where(e[..., None] == 122, np.clip(codes, -63, 63), codes)
    assert np.abs(codes).max(initial=0) <= 127
    return codes.astype(np.int8).reshape(rows, groups * 32), np.where(fine, e + 127, 255).astype(np.uint8)


def act8_decode(codes, scales, cols):
    rows, groups = scales.shape
    scale = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    return (codes.reshape(rows, groups, 32).astype(np.float64) * scale[..., None]).reshape(rows, groups * 32)[:, :cols]


def act8_buffer(codes, scales):
    """The checkpoint buffer as a device tensor."""
    return torch.from_numpy(np.concatenate([codes.view(np.uint8).reshape(-1), scales.reshape(-1)])).cuda()


def normals(seed, *shape, std=1.0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=F64) * std


def close(got, want, tol, what):
    """Every element of got within tol (a tensor or number) of want; equal where want is not finite."""
    got, want = got.double().cpu(), want.double().cpu()
    tol = torch.as_tensor(tol, dtype=F64).expand_as(want)
    odd = ~torch.isfinite(want)
    same = torch.where(torch.isnan(want), torch.isnan(got), got == want)
    bad = torch.where(odd, ~same, ~((got - want).abs() <= tol))
    if bad.any():
        i = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {i}: got {got[i]!r}, want {want[i]!r}, "
                             f"tolerance {float(tol[i]):.3g}")


def act_and_slope(g, act):
    """Activation and its derivative in 64 bits."""
    if act == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    cdf = 0.5 * torch.erfc(-g / math.sqrt(2))
    return g * cdf, cdf + g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)

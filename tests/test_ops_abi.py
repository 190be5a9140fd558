"""The training operators' C entries without a GPU: sizes, and refusals, which come before any CUDA call."""
import ctypes
import os
import shutil
import subprocess

import pytest

from fsdp2_gradient_packing_gb300 import _build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = ctypes.c_void_p(4096)       # a pointer that no refused call follows
ODD = ctypes.c_void_p(4098)


@pytest.fixture(scope="module")
def fp():
    import torch
    if torch.cuda.is_available():
        pytest.skip("made-up pointers: only where no kernel could run on them")
    _build.build()
    from fsdp2_gradient_packing_gb300 import fsdp_pack
    return fsdp_pack


def refused(fp, status, want, word):
    assert status == want, fp.fsdp_last_error()
    assert word in fp.fsdp_last_error()


@pytest.mark.parametrize("rows,cols,want", [(0, 1, 0), (1, 1, 33), (1, 32, 33), (1, 33, 66), (3, 4096, 3 * 4224), (7, 1409, 7 * 45 * 33),
                                            (1 << 20, 1 << 15, (1 << 20) * 33 * 1024)])
def test_act8_bytes(fp, rows, cols, want):
    assert fp.fsdp_act8_bytes(rows, cols) == want


def test_act8_refusals(fp):
    lib, out = fp._lib, ctypes.c_int64()
    E, U = fp.FSDP_EINVAL, fp.FSDP_EUNSUPPORTED
    refused(fp, lib.fsdp_act8_bytes(1, 1, None), E, "NULL")
    refused(fp, lib.fsdp_act8_bytes(-1, 1, ctypes.byref(out)), E, "rows")
    refused(fp, lib.fsdp_act8_bytes(1, 0, ctypes.byref(out)), E, "cols")
    refused(fp, lib.fsdp_act8_bytes(1 << 40, 1 << 40, ctypes.byref(out)), U, "too large")
    refused(fp, lib.fsdp_act8_store(P, 2, 4, 64, 64, P, None), E, "dtype")
    refused(fp, lib.fsdp_act8_store(P, 0, 4, 64, 63, P, None), E, "row distance")
    refused(fp, lib.fsdp_act8_store(None, 0, 4, 64, 64, P, None), E, "x is NULL")
    refused(fp, lib.fsdp_act8_store(ODD, 0, 4, 64, 64, P, None), E, "4-byte aligned")
    refused(fp, lib.fsdp_act8_store(P, 0, 4, 64, 64, ctypes.c_void_p(4104), None), E, "16-byte aligned")
    refused(fp, lib.fsdp_act8_load(P, 4, 64, None, 0, 64, None), E, "y is NULL")
    refused(fp, lib.fsdp_act8_load(P, -4, 64, P, 0, 64, None), E, "rows")
    assert lib.fsdp_act8_load(P, 0, 64, None, 0, 64, None) == fp.FSDP_OK


def norm(fp, **k):
    d = dict(rows=4, cols=64, ld_x=64, ld_y=64, ld_dx=64, x_dtype=1, y_dtype=1, dx_dtype=1, param_dtype=0, grad_dtype=0, eps=1e-5)
    d.update(k)
    return ctypes.byref(fp.fsdp_norm_desc_t(**d))


def test_norm_refusals(fp):
    lib = fp._lib
    E, U = fp.FSDP_EINVAL, fp.FSDP_EUNSUPPORTED

    def forward(d, x=P, w=P, b=P, y=P, m=P, r=P, keep=None):
        return lib.fsdp_layer_norm_forward(d, x, w, b, y, m, r, keep, None)

    refused(fp, forward(None), E, "desc")
    refused(fp, forward(norm(fp, rows=-1)), E, "rows")
    refused(fp, forward(norm(fp, cols=0)), E, "cols")
    refused(fp, forward(norm(fp, cols=65537, ld_x=65537, ld_y=65537)), U, "FSDP_NORM_MAX_COLS")
    refused(fp, forward(norm(fp, x_dtype=3)), E, "x_dtype")
    refused(fp, forward(norm(fp, y_dtype=2)), E, "y_dtype")
    refused(fp, forward(norm(fp, param_dtype=2)), E, "param_dtype")
    refused(fp, forward(norm(fp, eps=-1e-9)), E, "eps")
    refused(fp, forward(norm(fp, eps=float("inf"))), E, "eps")
    refused(fp, forward(norm(fp, ld_x=63)), E, "row distance")
    refused(fp, forward(norm(fp), x=None), E, "x is NULL")
    refused(fp, forward(norm(fp, x_dtype=2), x=ctypes.c_void_p(4104)), E, "16-byte")
    refused(fp, forward(norm(fp), y=None), E, "y is NULL")
    refused(fp, forward(norm(fp), w=ODD), E, "weight")
    refused(fp, forward(norm(fp), r=None), E, "together")
    refused(fp, forward(norm(fp, x_dtype=2), keep=P), E, "checkpoint already")
    assert forward(norm(fp, rows=0), x=None, y=None, m=None, r=None) == fp.FSDP_OK

    def backward(d, dy=P, x=P, w=P, m=P, r=P, dx=P, dw=P, db=P, ws=P, n=1 << 30):
        return lib.fsdp_layer_norm_backward(d, dy, x, w, m, r, dx, dw, db, ws, n, None)

    refused(fp, backward(norm(fp), dy=None), E, "dy is NULL")
    refused(fp, backward(norm(fp), m=None), E, "mean is NULL")
    refused(fp, backward(norm(fp, dx_dtype=5)), E, "dx_dtype")
    refused(fp, backward(norm(fp, grad_dtype=5)), E, "grad_dtype")
    refused(fp, backward(norm(fp, ld_dx=1)), E, "dx")
    refused(fp, backward(norm(fp, rows=4000), n=0), E, "workspace_bytes")
    refused(fp, backward(norm(fp, rows=4000), ws=ctypes.c_void_p(4104)), E, "workspace")
    refused(fp, backward(norm(fp, rows=4000), ws=None), E, "workspace is NULL")
    assert fp.fsdp_layer_norm_workspace(1000, 512) >= 2 * 512 * 4
    assert fp.fsdp_layer_norm_workspace(0, 512) == 0 and fp.fsdp_layer_norm_workspace(1, 512) == 0


def ffn(fp, **k):
    d = dict(rows=40, d=64, f=96, ld_x=64, ld_w_gate=64, ld_w_up=64, ld_h=96, ld_kept=96, ld_dx=64, ld_dw_gate=64, ld_dw_up=64,
             activation=0, keep=0, x_dtype=1, dx_dtype=1, dw_dtype=1, unaligned=0)
    d.update(k)
    return ctypes.byref(fp.fsdp_ffn_desc_t(**d))


def test_ffn_refusals(fp):
    lib = fp._lib
    E, U = fp.FSDP_EINVAL, fp.FSDP_EUNSUPPORTED

    def forward(d, x=P, g=P, u=P, h=P, kg=None, ku=None, ws=P, n=1 << 40):
        return lib.fsdp_gated_ffn_forward(d, x, g, u, h, kg, ku, ws, n, None)

    refused(fp, forward(None), E, "desc")
    refused(fp, forward(ffn(fp, rows=-1)), E, "rows")
    refused(fp, forward(ffn(fp, d=0)), E, "d < 1")
    refused(fp, forward(ffn(fp, rows=1 << 31)), U, "2^31")
    refused(fp, forward(ffn(fp, rows=(1 << 31) - 1024, f=(1 << 31) - 1024, ld_h=1 << 31)), U, "tiles")
    refused(fp, forward(ffn(fp, activation=2)), E, "activation")
    refused(fp, forward(ffn(fp, keep=3)), E, "keep")
    refused(fp, forward(ffn(fp, x_dtype=0)), U, "BF16")
    refused(fp, forward(ffn(fp, x_dtype=2)), E, "BF16")
    refused(fp, forward(ffn(fp, unaligned=8)), E, "unaligned")
    refused(fp, forward(ffn(fp, ld_w_up=63)), E, "w_up")
    refused(fp, forward(ffn(fp), g=None), E, "w_gate is NULL")
    refused(fp, forward(ffn(fp), x=ODD), E, "unaligned")
    refused(fp, forward(ffn(fp), kg=P), E, "FSDP_KEEP_NONE")
    refused(fp, forward(ffn(fp, keep=1), kg=P), E, "up is NULL")
    refused(fp, forward(ffn(fp, keep=2, ld_kept=95), kg=P, ku=P), E, "gate")
    refused(fp, forward(ffn(fp, ld_x=65), n=0), E, "workspace_bytes")
    assert forward(ffn(fp, rows=0), x=None, h=None) == fp.FSDP_OK

    def backward(d, dh=P, x=P, g=P, u=P, kg=None, ku=None, dx=P, dg=P, du=P, ws=P, n=1 << 40):
        return lib.fsdp_gated_ffn_backward(d, dh, x, g, u, kg, ku, dx, dg, du, ws, n, None)

    refused(fp, backward(ffn(fp), dh=None), E, "dh is NULL")
    refused(fp, backward(ffn(fp, x_dtype=2), x=ctypes.c_void_p(4104)), E, "16-byte")
    refused(fp, backward(ffn(fp, dx_dtype=2)), E, "dx_dtype")
    refused(fp, backward(ffn(fp, dw_dtype=2)), E, "dw_dtype")
    refused(fp, backward(ffn(fp), dg=None), E, "together")
    refused(fp, backward(ffn(fp, ld_dw_gate=1)), E, "dw_gate")
    refused(fp, backward(ffn(fp), n=0), E, "workspace_bytes")
    refused(fp, backward(ffn(fp), ws=None), E, "workspace is NULL")


def test_ffn_workspace(fp):
    """A forward call on aligned operands needs none; copies and the backward pass's dg and du are counted."""
    assert fp.fsdp_gated_ffn_workspace(1000, 64, 96, False) == 0
    assert fp.fsdp_gated_ffn_workspace(1000, 65, 96, False) >= 2 * (1000 + 2 * 96) * 72
    assert fp.fsdp_gated_ffn_workspace(1000, 64, 96, True) >= 2 * 2 * 1000 * 96
    assert fp.fsdp_gated_ffn_workspace(1000, 64, 96, True, x_act8=True) >= 2 * 2 * 1000 * 96 + 2 * 1000 * 64
    assert fp.fsdp_gated_ffn_workspace(0, 64, 96, True) == 0


@pytest.mark.parametrize("backward,x_act8", [(False, False), (True, False), (True, True)])
@pytest.mark.parametrize("rows,d,f", [(1, 64, 96), (5, 64, 96), (1000, 64, 96), (1000, 65, 96), (129, 512, 1408)])
def test_ffn_workspace_of_views(fp, rows, d, f, backward, x_act8):
    """What the binding gives for operands that are not aligned is enough for every row distance and offset of each."""
    bound = fp.fsdp_gated_ffn_workspace(rows, d, f, backward, x_act8=x_act8, aligned=False)
    assert bound >= fp.fsdp_gated_ffn_workspace(rows, d, f, backward, x_act8=x_act8)
    out = ctypes.c_int64()
    for off in range(8):
        for lx, lg, lu in ((0, 0, 0), (1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 3, 5), (8, 8, 8)):
            desc = ffn(fp, rows=rows, d=d, f=f, ld_x=d + lx, ld_w_gate=d + lg, ld_w_up=d + lu, ld_h=f, ld_kept=f, ld_dx=d,
                       ld_dw_gate=d, ld_dw_up=d, x_dtype=2 if x_act8 else 1, unaligned=off)
            assert fp._lib.fsdp_gated_ffn_workspace(desc, int(backward), ctypes.byref(out)) == fp.FSDP_OK
            assert out.value <= bound


def test_binding_checks_without_tensors_on_a_gpu(fp):
    import torch
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError, match="not a CUDA tensor"):
        fp.fsdp_layer_norm_forward(x, None, None, x)
    with pytest.raises(ValueError, match="3 dimensions"):
        fp.fsdp_act8_store(torch.zeros(1, 2, 3), None)
    with pytest.raises(ValueError, match="not a tensor"):
        fp.fsdp_act8_store([1.0], None)
    with pytest.raises(ValueError, match="no checkpoint"):
        fp.Act8(4, 0)


def test_header_in_strict_c(tmp_path):
    if not shutil.which("gcc"):
        pytest.skip("gcc is not installed")
    src = tmp_path / "ops.c"
    src.write_text('#include "fsdp_ops.h"\nint main(void) { fsdp_norm_desc_t n; fsdp_ffn_desc_t f; (void)&n; (void)&f; '
                   'return sizeof n == 64 && sizeof f == 112 ? 0 : 1; }\n')
    exe = tmp_path / "ops"
    subprocess.run(["gcc", "-std=c99", "-pedantic", "-Wall", "-Wextra", "-Werror", "-I", os.path.join(ROOT, "include"), str(src),
                    "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)]).returncode == 0

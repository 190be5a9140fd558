"""8-bit activation checkpoints: codes, scale bytes and values read back equal the definition bit for bit."""
import numpy as np
import pytest
import torch

from gpu_util import fp_module
from ops_util import BF16, F32, Matrix, act8_buffer, act8_decode, act8_encode, normals

pytestmark = pytest.mark.gpu


def _values(rows, cols, dtype, seed):
    x = normals(seed, rows, cols).float()
    x *= 2.0 ** (torch.arange(cols) % 61 - 30.0)  # groups of very different size
    return x.to(dtype)


def _round_trip(fp, m, dtype):
    rows, cols = m.t.shape
    n = fp.fsdp_act8_bytes(rows, cols)
    assert n == rows * 33 * ((cols + 31) // 32)
    buf = torch.full((n + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    ck = fp.Act8(rows, cols, buf)
    fp.fsdp_act8_store(m.t, ck)
    groups = (cols + 31) // 32
    raw = buf.cpu().numpy()
    assert (raw[n:] == 0xA5).all()
    codes = raw[:rows * groups * 32].view(np.int8).reshape(rows, groups * 32)
    scales = raw[rows * groups * 32:n].reshape(rows, groups)
    want_codes, want_scales = act8_encode(m.t.double().cpu().numpy())
    assert np.array_equal(scales, want_scales)
    assert np.array_equal(codes, want_codes)
    want = act8_decode(want_codes, want_scales, cols)
    for out in (F32, BF16):
        y = Matrix(rows, cols, out, m.ld, 0)
        fp.fsdp_act8_load(ck, y.t)
        got = y.t.double().cpu().numpy()
        assert np.array_equal(got, want, equal_nan=True), out
        assert y.intact()
    # Storing what was read back gives the same checkpoint.
    y = torch.empty(rows, cols, dtype=dtype, device="cuda")
    fp.fsdp_act8_load(ck, y)
    again = fp.Act8(rows, cols)
    fp.fsdp_act8_store(y, again)
    back = torch.empty_like(y)
    fp.fsdp_act8_load(again, back)
    assert torch.equal(torch.nan_to_num(back, 7.0), torch.nan_to_num(y, 7.0))
    assert m.intact()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 7), (1, 31), (5, 32), (4, 33), (257, 64), (2, 100), (9, 1409), (33, 4096),
                                       (1025, 40), (65, 12288)])
def test_round_trip(rows, cols, dtype):
    _round_trip(fp_module(), Matrix(rows, cols, dtype, value=_values(rows, cols, dtype, rows * cols)), dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("cols,ld,offset", [(64, 64, 1), (64, 72, 0), (64, 65, 0), (40, 48, 8), (33, 40, 0), (8, 8, 3)])
def test_strides_and_offsets(cols, ld, offset, dtype):
    _round_trip(fp_module(), Matrix(21, cols, dtype, ld, offset, _values(21, cols, dtype, ld)), dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("cols", [96, 99])
def test_special_values(cols, dtype):
    big = torch.finfo(dtype).max
    x = torch.zeros(12, cols, dtype=torch.float64)
    x[1, 5] = float("nan")
    x[2, 40] = float("inf")
    x[3, 95] = float("-inf")
    x[4, :40] = big
    x[5, :] = -big / 3
    x[6, :] = 2.0 ** -130      # subnormal in both types
    x[7, :] = 2.0 ** -126
    x[8, :50] = 127 * 2.0 ** -3            # exactly at the border of a scale
    x[9, :32] = torch.arange(32) + 0.5     # ties
    x[9, 31] = 127
    x[10, :] = -0.0
    x[11, :] = 128
    _round_trip(fp_module(), Matrix(12, cols, dtype, value=x.to(dtype).double()), dtype)


@pytest.mark.parametrize("k", range(0, 512, 64))
def test_borders_of_a_scale(k):
    """FP32 tops around the largest magnitude that a scale holds, 127 * 2^e, one ulp to each side."""
    base = torch.tensor([127 * 2.0 ** (k / 4 - 100)]).float()
    tops = torch.cat([base, torch.nextafter(base, base * 2), torch.nextafter(base, base * 0)])
    x = normals(k, 3, 32).float().clamp(-1, 1) * tops[:, None] * 0.99
    x[:, 7] = tops
    _round_trip(fp_module(), Matrix(3, 32, F32, value=x), F32)


def test_views_read_what_they_cover():
    fp = fp_module()
    ck, _ = act8_encode(np.ones((2, 32))), None
    a = fp.Act8(2, 32, act8_buffer(*ck))
    y = torch.empty(2, 32, device="cuda")
    fp.fsdp_act8_load(a, y)
    assert bool((y == 1).all())


def test_refusals():
    fp = fp_module()
    x = torch.zeros(4, 64, device="cuda")
    with pytest.raises(ValueError, match="checkpoint of 4 x 32"):
        fp.fsdp_act8_store(x, fp.Act8(4, 32))
    with pytest.raises(ValueError, match="column stride"):
        fp.fsdp_act8_store(torch.zeros(64, 4, device="cuda").t(), fp.Act8(4, 64))
    with pytest.raises(ValueError, match="elements apart"):
        fp.fsdp_act8_store(torch.zeros(1, 64, device="cuda").expand(4, 64), fp.Act8(4, 64))
    with pytest.raises(ValueError, match="float16"):
        fp.fsdp_act8_load(fp.Act8(4, 64), torch.zeros(4, 64, device="cuda", dtype=torch.float16))
    with pytest.raises(ValueError, match="not a CUDA tensor"):
        fp.fsdp_act8_store(torch.zeros(4, 64), fp.Act8(4, 64))
    with pytest.raises(ValueError, match="at least 132 bytes"):
        fp.Act8(4, 32, torch.empty(100, dtype=torch.uint8, device="cuda"))
    data = torch.empty(4 * 66 + 8, dtype=torch.uint8, device="cuda")[8:]
    with pytest.raises(fp.FsdpError, match="16-byte"):
        fp.fsdp_act8_store(x, fp.Act8(4, 64, data))


def test_empty_matrix():
    fp = fp_module()
    fp.fsdp_act8_store(torch.zeros(0, 64, device="cuda"), fp.Act8(0, 64))
    fp.fsdp_act8_load(fp.Act8(0, 64), torch.zeros(0, 64, device="cuda"))

"""Layer norm against its definition in 64 bits.

Tolerances.  In units u = 2^-24: a sum of n values runs in per-thread chains of at most 16 terms and then a tree or chain
of at most 16 + 5 + 16 + 8 more, so its error is at most 64 u times the sum of magnitudes.  With S = max|x| over the
row, the mean is off by at most 64 u S, xh by 64 u S rstd more than its own few roundings, and rstd (from squares that
shift by the mean's error only in second order) by 64 u relative.  A result in a narrower type adds half an ulp of it.
"""
import pytest
import torch

from gpu_util import fp_module
from ops_util import BF16, EPS32, F32, F64, HALF, Matrix, act8_buffer, act8_decode, act8_encode, close, normals

pytestmark = pytest.mark.gpu
U = 64 * EPS32


def reference(x, w, b, eps):
    mean = x.mean(-1)
    xc = x - mean[:, None]
    rstd = 1 / torch.sqrt(xc.square().mean(-1) + eps)
    y = xc * rstd[:, None]
    y = y if w is None else y * w
    return (y if b is None else y + b), mean, rstd


def check_forward(fp, x, w, b, y_dtype, ld=None, offset=0, eps=1e-5, keep=False, from_ckpt=False):
    """x, w, b: CPU tensors in their dtypes."""
    rows, cols = x.shape
    mx = Matrix(rows, cols, x.dtype, ld, offset, x)
    my = Matrix(rows, cols, y_dtype, ld, offset)
    dw, db = (None if t is None else t.cuda() for t in (w, b))
    mean, rstd = torch.full((rows,), 9.0, device="cuda"), torch.full((rows,), 9.0, device="cuda")
    kept = fp.Act8(rows, cols) if keep else None
    x64 = x.double()
    src = mx.t
    if from_ckpt:
        enc = act8_encode(x64.numpy())
        src = fp.Act8(rows, cols, act8_buffer(*enc))
        x64 = torch.from_numpy(act8_decode(*enc, cols))
    fp.fsdp_layer_norm_forward(src, dw, db, my.t, mean, rstd, eps=eps, keep=kept)
    y64, m64, r64 = reference(x64, None if w is None else w.double(), None if b is None else b.double(), eps)
    top = x64.abs().amax(-1)
    close(mean, m64, U * top + 1e-40, "mean")
    close(rstd, r64, U * r64 * (1 + top * r64), "rstd")
    size = (w.double().abs() if w is not None else torch.ones(cols, dtype=F64))
    off = U * (2 + (top * r64)[:, None] * 2 + ((x64 - m64[:, None]) * r64[:, None]).abs()) * size
    close(my.t, y64, off * (1 + top * r64)[:, None].clamp(max=4) + (y64.abs() + off) * HALF[y_dtype], "y")
    assert mx.intact() and my.intact()
    if keep:
        codes, scales = act8_encode(x.double().numpy())
        assert torch.equal(kept.data.cpu(), act8_buffer(codes, scales).cpu())


def make(rows, cols, seed, dtype=F32, pdtype=F32, shift=0.2):
    x = (normals(seed, rows, cols) * (0.5 + normals(seed + 1, cols).abs()) + shift).to(dtype)
    return x, (1 + normals(seed + 2, cols, std=0.2)).to(pdtype), normals(seed + 3, cols, std=0.2).to(pdtype)


WIDTHS = [1, 2, 8, 31, 40, 256, 511, 512, 520, 1000, 1024, 1409, 2048, 2056, 4096, 5001, 8192, 8200, 9001, 16384, 20000,
          40008]


@pytest.mark.parametrize("dtype,y_dtype", [(BF16, BF16), (F32, F32), (F32, BF16), (BF16, F32)])
@pytest.mark.parametrize("cols", WIDTHS)
def test_forward(cols, dtype, y_dtype):
    fp = fp_module()
    x, w, b = make(7, cols, cols, dtype)
    check_forward(fp, x, w, b, y_dtype, keep=True)
    check_forward(fp, x, w, b, y_dtype, from_ckpt=True)


@pytest.mark.parametrize("rows", [1, 2, 5, 4099])
@pytest.mark.parametrize("cols", [96, 1409])
def test_forward_rows(rows, cols):
    x, w, b = make(rows, cols, rows, BF16, BF16)
    check_forward(fp_module(), x, w, b, BF16, keep=True)


@pytest.mark.parametrize("ld,offset", [(64, 1), (72, 0), (65, 0), (64, 8)])
def test_forward_strides(ld, offset):
    x, w, b = make(9, 64, ld, BF16)
    check_forward(fp_module(), x, w, b, BF16, ld, offset, keep=True)
    check_forward(fp_module(), x.float(), w, None, F32, ld, offset)
    check_forward(fp_module(), x, None, b, F32, ld, offset)
    check_forward(fp_module(), x, None, None, BF16, ld, offset)


def test_unaligned_parameters():
    fp = fp_module()
    x, w, b = make(3, 64, 5)
    y = torch.empty(3, 64, device="cuda")
    wide = torch.zeros(65, device="cuda")
    wide[1:] = w
    fp.fsdp_layer_norm_forward(x.cuda(), wide[1:], b.cuda(), y)
    close(y, reference(x.double(), w.double(), b.double(), 1e-5)[0], 1e-4, "y")


def test_large_mean_keeps_its_variance():
    """Rows far from 0: the variance comes from differences, not from a difference of squares."""
    x = (normals(3, 6, 4096) + 3000).float()
    check_forward(fp_module(), x, None, None, F32)


def test_constant_and_special_rows():
    fp = fp_module()
    x = torch.ones(6, 96)
    x[1] = 0
    x[2, 5] = float("nan")
    x[3, 50] = float("inf")
    x[4] = torch.linspace(-1, 1, 96)
    y, mean, rstd = torch.empty(6, 96, device="cuda"), torch.empty(6, device="cuda"), torch.empty(6, device="cuda")
    fp.fsdp_layer_norm_forward(x.cuda(), None, None, y, mean, rstd)
    assert bool((y[:2] == 0).all()) and bool(torch.isnan(y[2:4]).all()) and bool(torch.isfinite(y[4:]).all())
    # eps 0 on a constant row: 0 * infinity, in that row alone.
    fp.fsdp_layer_norm_forward(x.cuda(), None, None, y, mean, rstd, eps=0.0)
    assert bool(torch.isnan(y[:2]).all()) and bool(torch.isfinite(y[4]).all())


def backward_reference(x, w, dy, mean, rstd):
    xh = (x - mean[:, None]) * rstd[:, None]
    g = dy if w is None else dy * w
    c1, c2 = (g * xh).mean(-1, keepdim=True), g.mean(-1, keepdim=True)
    return rstd[:, None] * (g - c2 - xh * c1), (dy * xh).sum(0), dy.sum(0), xh, g, c1, c2


def check_backward(fp, x, w, dy, dx_dtype, grad_dtype=F32, ld=None, offset=0, from_ckpt=False, want=(True, True, True)):
    rows, cols = x.shape
    x64 = x.double()
    _, m64, r64 = reference(x64, None, None, 1e-5)
    mean, rstd = m64.float(), r64.float()
    src = Matrix(rows, cols, x.dtype, ld, offset, x)
    arg = src.t
    if from_ckpt:
        enc = act8_encode(x64.numpy())
        arg, x64 = fp.Act8(rows, cols, act8_buffer(*enc)), torch.from_numpy(act8_decode(*enc, cols))
    mdy = Matrix(rows, cols, dy.dtype, ld, offset, dy)
    mdx = Matrix(rows, cols, dx_dtype, ld, offset)
    grads = [Matrix(1, cols, grad_dtype, None, offset) for _ in range(2)]
    fp.fsdp_layer_norm_backward(mdy.t, arg, None if w is None else w.cuda(), mean.cuda(), rstd.cuda(),
                                mdx.t if want[0] else None, grads[0].t if want[1] else None,
                                grads[1].t if want[2] else None)
    dx, dw, db, xh, g, c1, c2 = backward_reference(x64, None if w is None else w.double(), dy.double(), mean.double(),
                                                   rstd.double())
    if want[0]:
        parts = g.abs() + g.abs().mean(-1, keepdim=True) + xh.abs() * (g * xh).abs().mean(-1, keepdim=True)
        off = U * rstd.double()[:, None] * parts * (1 + (x64.abs().amax(-1) * rstd.double())[:, None].clamp(max=64))
        close(mdx.t, dx, off + (dx.abs() + off) * HALF[dx_dtype], "dx")
    chain = (64 + rows / 100) * EPS32  # terms that one thread, then one warp, adds in a chain
    for on, got, ref, size, what in ((want[1], grads[0].t[0], dw, (dy.double() * xh).abs().sum(0), "dweight"),
                                     (want[2], grads[1].t[0], db, dy.double().abs().sum(0), "dbias")):
        if on:
            off = chain * size + (U * (x64.abs().amax(-1, keepdim=True) * rstd.double()[:, None]) * dy.double().abs()).sum(0)
            close(got, ref, off + (ref.abs() + off) * HALF[grad_dtype], what)
    assert src.intact() and mdy.intact() and mdx.intact() and all(m.intact() for m in grads)


@pytest.mark.parametrize("dtype,y_dtype,dx_dtype", [(BF16, BF16, BF16), (F32, F32, F32), (F32, BF16, F32), (BF16, F32, BF16)])
@pytest.mark.parametrize("cols", WIDTHS)
def test_backward(cols, dtype, y_dtype, dx_dtype):
    fp = fp_module()
    x, w, _ = make(13, cols, cols + 1, dtype)
    dy = normals(cols, 13, cols, std=0.01).to(y_dtype)
    check_backward(fp, x, w, dy, dx_dtype)
    check_backward(fp, x, w, dy, dx_dtype, BF16, from_ckpt=True)


@pytest.mark.parametrize("shift,std", [(3000.0, 1.0), (100.0, 0.01)])
@pytest.mark.parametrize("from_ckpt", [False, True])
@pytest.mark.parametrize("cols", [96, 99, 1024, 2048, 4104, 5001, 9000])
def test_backward_far_from_zero(cols, from_ckpt, shift, std):
    """Rows whose mean is many times their deviation, and a constant row, whose xh is 0.  xh is a difference rounded once
    and a product rounded once, so its error is 2 u of xh itself, whatever the mean: dx is then within the sums' 64 u of its
    terms, and dweight within its chains' of the terms' magnitudes."""
    fp = fp_module()
    rows = 40
    x = (normals(cols, rows, cols, std=std) + shift).float()
    x[7] = shift + 1.3
    w, dy = (1 + normals(1, cols, std=0.2)).float(), normals(2, rows, cols).float()
    x64 = x.double()
    _, m64, r64 = reference(x64, None, None, 1e-5)
    mean, rstd = m64.float(), r64.float()
    arg = x.cuda()
    if from_ckpt:
        enc = act8_encode(x64.numpy())
        arg, x64 = fp.Act8(rows, cols, act8_buffer(*enc)), torch.from_numpy(act8_decode(*enc, cols))
    dx, dw, db = torch.empty(rows, cols, device="cuda"), torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    fp.fsdp_layer_norm_backward(dy.cuda(), arg, w.cuda(), mean.cuda(), rstd.cuda(), dx, dw, db)
    dx64, dw64, db64, xh, g, _, _ = backward_reference(x64, w.double(), dy.double(), mean.double(), rstd.double())
    assert from_ckpt or bool((xh[7] == 0).all())
    parts = g.abs() + g.abs().mean(-1, keepdim=True) + 2 * xh.abs() * (g * xh).abs().mean(-1, keepdim=True)
    close(dx, dx64, U * rstd.double()[:, None] * parts, "dx")
    close(dw, dw64, U * (dy.double() * xh).abs().sum(0), "dweight")
    close(db, db64, U * dy.double().abs().sum(0), "dbias")


@pytest.mark.parametrize("rows", [1, 2, 5, 1000, 9001])
@pytest.mark.parametrize("cols", [96, 99, 1024])
def test_backward_rows(rows, cols):
    x, w, _ = make(rows, cols, rows, BF16, BF16)
    dy = normals(rows, rows, cols).to(BF16)
    check_backward(fp_module(), x, w, dy, F32)
    check_backward(fp_module(), x, w, dy, BF16, from_ckpt=True)


@pytest.mark.parametrize("cols", [8208, 9001, 17000])
@pytest.mark.parametrize("rows", [155, 1000])
def test_wide_rows_in_turns(rows, cols):
    """Clusters with several rows at a time, the last turn with rows for some of them."""
    fp = fp_module()
    x, w, b = make(rows, cols, cols + rows, BF16)
    check_forward(fp, x, w, b, BF16, keep=True)
    check_forward(fp, x, w, b, F32, from_ckpt=True)
    check_backward(fp, x, w, normals(rows, rows, cols).to(BF16), BF16)
    check_backward(fp, x, w, normals(rows, rows, cols).to(BF16), BF16, from_ckpt=True)


@pytest.mark.parametrize("ld,offset", [(64, 1), (72, 0), (65, 0), (64, 8)])
def test_backward_strides(ld, offset):
    x, w, _ = make(9, 64, ld, BF16)
    dy = normals(ld, 9, 64).to(BF16)
    check_backward(fp_module(), x, w, dy, BF16, BF16, ld, offset)
    check_backward(fp_module(), x.float(), None, dy.float(), F32, F32, ld, offset)


@pytest.mark.parametrize("want", [(True, False, False), (False, True, False), (False, False, True), (False, True, True)])
@pytest.mark.parametrize("rows,cols", [(3, 96), (700, 96), (700, 2048)])
def test_backward_parts(rows, cols, want):
    x, w, _ = make(rows, cols, 2)
    check_backward(fp_module(), x, w, normals(3, rows, cols).float(), F32, want=want)


@pytest.mark.parametrize("cols", [48, 1409, 9000])
def test_gradient_against_differences(cols):
    """Directional derivatives of sum(dy * y) with y from 64-bit arithmetic.  The central difference is off by its third
    derivative times h^2 / 6 (below 1e-9 relative at h = 1e-5) and by rounding (1e-16 / h), the kernel by its own
    binary32 sums: 1e-5 of the sum of magnitudes covers both."""
    fp = fp_module()
    rows, h = 5, 1e-5
    x, w, b = make(rows, cols, 11)
    dy = normals(12, rows, cols).float()
    y, mean, rstd = torch.empty(rows, cols, device="cuda"), torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    fp.fsdp_layer_norm_forward(x.cuda(), w.cuda(), b.cuda(), y, mean, rstd)
    dx, dw, db = torch.empty_like(y), torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    fp.fsdp_layer_norm_backward(dy.cuda(), x.cuda(), w.cuda(), mean, rstd, dx, dw, db)

    def loss(x, w, b):
        return float((dy.double() * reference(x, w, b, 1e-5)[0]).sum())

    args = [x.double(), w.double(), b.double()]
    for k, grad in enumerate((dx, dw, db)):
        v = normals(20 + k, *args[k].shape)
        hi, lo = [a.clone() for a in args], [a.clone() for a in args]
        hi[k] += h * v
        lo[k] -= h * v
        diff = (loss(*hi) - loss(*lo)) / (2 * h)
        terms = grad.double().cpu() * v
        assert abs(float(terms.sum()) - diff) <= 1e-5 * float(terms.abs().sum()) + 1e-8


def test_no_rows():
    fp = fp_module()
    e = torch.empty(0, 64, device="cuda")
    m = torch.empty(0, device="cuda")
    w = torch.ones(64, device="cuda")
    fp.fsdp_layer_norm_forward(e, w, w, e, m, m)
    dw, db = torch.full((64,), 7.0, device="cuda"), torch.full((64,), 7.0, device="cuda")
    fp.fsdp_layer_norm_backward(e, e, w, m, m, e, dw, db)
    assert bool((dw == 0).all()) and bool((db == 0).all())


def test_same_bits_on_every_run_and_stream():
    fp = fp_module()
    x, w, _ = make(3000, 1024, 4, BF16)
    dy = normals(5, 3000, 1024).to(BF16).cuda()
    x, w = x.cuda(), w.cuda()
    mean, rstd = x.float().mean(-1), torch.ones(3000, device="cuda")
    torch.cuda.synchronize()
    outs = []
    side = torch.cuda.Stream()
    for stream in (None, side, side, None):
        dx, dw, db = torch.empty_like(dy), torch.empty_like(w), torch.empty_like(w)
        torch.cuda.synchronize()
        fp.fsdp_layer_norm_backward(dy, x, w, mean, rstd, dx, dw, db, stream=stream)
        torch.cuda.synchronize()
        outs.append((dx, dw, db))
    for o in outs[1:]:
        assert all(torch.equal(p, q) for p, q in zip(o, outs[0]))


def test_refusals():
    fp = fp_module()
    x, w = torch.zeros(4, 64, device="cuda"), torch.ones(64, device="cuda")
    m = torch.zeros(4, device="cuda")
    with pytest.raises(ValueError, match="not 4 x 64"):
        fp.fsdp_layer_norm_forward(x[:, :32], w, w, x)
    with pytest.raises(ValueError, match="vector of 64"):
        fp.fsdp_layer_norm_forward(x, w[:32], None, torch.empty_like(x))
    with pytest.raises(ValueError, match="together"):
        fp.fsdp_layer_norm_forward(x, w, w, torch.empty_like(x), mean=m)
    with pytest.raises(ValueError, match="different dtypes"):
        fp.fsdp_layer_norm_forward(x, w, w.bfloat16(), torch.empty_like(x))
    with pytest.raises(fp.FsdpError, match="eps"):
        fp.fsdp_layer_norm_forward(x, w, w, torch.empty_like(x), eps=-1.0)
    with pytest.raises(fp.FsdpError, match="eps"):
        fp.fsdp_layer_norm_forward(x, w, w, torch.empty_like(x), eps=float("nan"))
    with pytest.raises(fp.FsdpError, match="checkpoint already"):
        fp.fsdp_layer_norm_forward(fp.Act8(4, 64), w, w, torch.empty_like(x), keep=fp.Act8(4, 64))
    with pytest.raises(ValueError, match="needed"):
        fp.fsdp_layer_norm_backward(x, x, w, m, None, torch.empty_like(x))
    many, rows = torch.zeros(4000, 64, device="cuda"), torch.zeros(4000, device="cuda")  # 4 rows need no workspace
    with pytest.raises(ValueError, match="the call needs"):
        fp.fsdp_layer_norm_backward(many, many, w, rows, rows, torch.empty_like(many),
                                    workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    wide = torch.zeros(1, 65537, device="cuda")
    with pytest.raises(fp.FsdpError, match="FSDP_NORM_MAX_COLS"):
        fp.fsdp_layer_norm_forward(wide, None, None, torch.empty_like(wide))

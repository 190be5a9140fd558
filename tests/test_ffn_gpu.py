"""Gated feed-forward block against its definition in 64 bits.

Tolerances.  A product of BF16 operands is exact in binary32; a sum of k of them, in whatever order and with each
addition rounded or cut to binary32, is off by at most k 2^-23 times the sum of magnitudes.  For g and u that is
E = d 2^-23 (|x| |W|^T).  The activations' own arithmetic adds 2^-18 relative (fast exponential and division: a few ulp,
|g| 2^-22 through the exponent).  Both act and its slope change by at most 1.2 times a change of g (|act'| <= 1.13,
|act''| <= 0.8 for both activations).  dg and du are rounded to BF16 (2^-8 relative) before the backward products,
whose error is then at most the product of those bounds with the other operand's magnitudes.  What is kept in 8 bits is
exactly the definition's for the checkpoint that the call was given; results in BF16 add half an ulp.
"""
import numpy as np
import pytest
import torch

from gpu_util import fp_module
from ops_util import (BF16, F32, F64, HALF, Matrix, act8_buffer, act8_decode, act8_encode, act_and_slope, close, normals)

pytestmark = pytest.mark.gpu
CUT = 2.0 ** -23
FAST = 2.0 ** -18


class Block:
    """Operands of one block, on the CPU in 64 bits (values exact in BF16) and on the GPU with strides and offsets."""

    def __init__(self, rows, d, f, seed=0, pad=0, offset=0):
        self.rows, self.d, self.f = rows, d, f
        self.x = normals(seed, rows, d).to(BF16).double()
        self.wg, self.wu = (normals(seed + k, f, d, std=d ** -0.5).to(BF16).double() for k in (1, 2))
        self.dh = normals(seed + 3, rows, f, std=0.1).to(BF16).double()
        self.mx = Matrix(rows, d, BF16, d + pad, offset, self.x)
        self.mwg, self.mwu = (Matrix(f, d, BF16, d + pad, offset, w) for w in (self.wg, self.wu))
        self.mdh = Matrix(rows, f, BF16, f + pad, offset, self.dh)
        self.pad, self.offset = pad, offset

    def out(self, rows, cols, dtype):
        return Matrix(rows, cols, dtype, cols + self.pad, self.offset)

    def gate_up(self):
        """g, u and the bounds of their errors."""
        g, u = self.x @ self.wg.T, self.x @ self.wu.T
        eg, eu = (self.d * CUT * (self.x.abs() @ w.abs().T) for w in (self.wg, self.wu))
        return g, u, eg, eu

    def intact(self):
        return all(m.intact() for m in (self.mx, self.mwg, self.mwu, self.mdh))


ACTS = {"silu": 0, "gelu": 1}


def check_forward(fp, b, act, keep):
    h = b.out(b.rows, b.f, BF16)
    gate = up = None
    if keep == "act8":
        gate, up = fp.Act8(b.rows, b.f), fp.Act8(b.rows, b.f)
    elif keep == "bf16":
        mg, mu = b.out(b.rows, b.f, BF16), b.out(b.rows, b.f, BF16)
        gate, up = mg.t, mu.t
    fp.fsdp_gated_ffn_forward(b.mx.t, b.mwg.t, b.mwu.t, h.t, gate=gate, up=up, activation=ACTS[act])
    fp.fsdp_ops_sync_status()
    g, u, eg, eu = b.gate_up()
    a, _ = act_and_slope(g, act)
    ea = 1.2 * eg + FAST * a.abs() + 1e-30
    off = ea * u.abs() + a.abs() * eu + ea * eu
    close(h.t, a * u, off + (a * u).abs() * HALF[BF16] + off * HALF[BF16], "h")
    assert h.intact() and b.intact()
    if keep == "bf16":
        close(mg.t, g, eg + (g.abs() + eg) * HALF[BF16], "gate")
        close(mu.t, u, eu + (u.abs() + eu) * HALF[BF16], "up")
        assert mg.intact() and mu.intact()
    elif keep == "act8":
        for ck, v, e in ((gate, g, eg), (up, u, eu)):
            y = torch.empty(b.rows, b.f, device="cuda")
            fp.fsdp_act8_load(ck, y)
            # At most half a step of the scale, which is below top / 63; e may move the top over a border.
            pad = torch.zeros(b.rows, (b.f + 31) // 32 * 32, dtype=F64)
            pad[:, :b.f] = v.abs() + e
            top = pad.view(b.rows, -1, 32).amax(-1).repeat_interleave(32, 1)[:, :b.f]
            close(y, v, e + top / 63 / 2, "kept")


def check_backward(fp, b, act, keep, x_act8=False, dx_dtype=BF16, dw_dtype=BF16, want=(True, True)):
    x, src = b.x, b.mx.t
    if x_act8:
        enc = act8_encode(b.x.numpy())
        x, src = torch.from_numpy(act8_decode(*enc, b.d)), fp.Act8(b.rows, b.d, act8_buffer(*enc))
    gate = up = None
    if keep == "none":
        g, u = x @ b.wg.T, x @ b.wu.T
        eg, eu = (b.d * CUT * (x.abs() @ w.abs().T) for w in (b.wg, b.wu))
    else:
        g, u = b.x @ b.wg.T, b.x @ b.wu.T
        eg = eu = torch.zeros_like(g)
        if keep == "act8":
            encs = [act8_encode(t.numpy()) for t in (g, u)]
            g, u = (torch.from_numpy(act8_decode(*e, b.f)) for e in encs)
            gate, up = (fp.Act8(b.rows, b.f, act8_buffer(*e)) for e in encs)
        else:
            g, u = g.to(BF16).double(), u.to(BF16).double()
            mg, mu = b.out(b.rows, b.f, BF16), b.out(b.rows, b.f, BF16)
            mg.t.copy_(g)
            mu.t.copy_(u)
            gate, up = mg.t, mu.t
    mdx, mdg, mdu = b.out(b.rows, b.d, dx_dtype), b.out(b.f, b.d, dw_dtype), b.out(b.f, b.d, dw_dtype)
    fp.fsdp_gated_ffn_backward(b.mdh.t, src, b.mwg.t, b.mwu.t, mdx.t if want[0] else None, mdg.t if want[1] else None,
                               mdu.t if want[1] else None, gate=gate, up=up, activation=ACTS[act])
    fp.fsdp_ops_sync_status()
    a, s = act_and_slope(g, act)
    dg, du = b.dh * u * s, b.dh * a
    es, ea = 1.2 * eg + FAST * (1 + g.abs()) + 1e-30, 1.2 * eg + FAST * a.abs() + 1e-30
    edg = b.dh.abs() * (u.abs() * es + s.abs() * eu + es * eu)
    edu = b.dh.abs() * ea
    edg, edu = (e + (v.abs() + e) * 2.0 ** -8 for e, v in ((edg, dg), (edu, du)))
    if want[0]:
        dx = dg @ b.wg + du @ b.wu
        size = (dg.abs() + edg) @ b.wg.abs() + (du.abs() + edu) @ b.wu.abs()
        off = edg @ b.wg.abs() + edu @ b.wu.abs() + 2 * (b.f + 64) * CUT * size
        close(mdx.t, dx, off + (dx.abs() + off) * HALF[dx_dtype], "dx")
    if want[1]:
        for m, v, e, what in ((mdg, dg, edg, "dw_gate"), (mdu, du, edu, "dw_up")):
            dw = v.T @ x
            off = e.T @ x.abs() + (b.rows + 64) * CUT * ((v.abs() + e).T @ x.abs())
            close(m.t, dw, off + (dw.abs() + off) * HALF[dw_dtype], what)
    assert b.intact() and mdx.intact() and mdg.intact() and mdu.intact()


SIZES = [(1, 1, 1), (1, 64, 64), (1, 512, 1408), (3, 7, 5), (5, 200, 33), (8, 72, 136), (9, 72, 136), (16, 16, 16),
         (33, 515, 257), (64, 64, 64), (65, 1000, 96), (127, 96, 300), (128, 128, 128), (129, 136, 257), (200, 512, 1408),
         (256, 256, 256), (257, 64, 513), (300, 40, 1000), (700, 1024, 520), (1025, 515, 131)]


@pytest.mark.parametrize("keep", ["none", "act8", "bf16"])
@pytest.mark.parametrize("rows,d,f", SIZES)
def test_forward(rows, d, f, keep):
    check_forward(fp_module(), Block(rows, d, f, rows + d + f), "silu" if rows % 2 else "gelu", keep)


@pytest.mark.parametrize("keep", ["none", "act8", "bf16"])
@pytest.mark.parametrize("rows,d,f", SIZES)
def test_backward(rows, d, f, keep):
    fp = fp_module()
    b = Block(rows, d, f, rows + d + f)
    check_backward(fp, b, "gelu" if rows % 2 else "silu", keep)
    check_backward(fp, b, "silu" if rows % 2 else "gelu", keep, x_act8=True, dx_dtype=F32, dw_dtype=F32)


@pytest.mark.parametrize("pad,offset", [(0, 1), (8, 0), (1, 0), (3, 5), (0, 8)])
@pytest.mark.parametrize("rows,d,f", [(130, 72, 136), (7, 65, 40)])
def test_strides_and_offsets(rows, d, f, pad, offset):
    fp = fp_module()
    b = Block(rows, d, f, 3, pad, offset)
    for keep in ("none", "act8", "bf16"):
        check_forward(fp, b, "silu", keep)
        check_backward(fp, b, "silu", keep, dw_dtype=F32)


@pytest.mark.parametrize("rows,d,f", [(64, 64, 16384), (40, 2048, 2048), (8192, 64, 64), (2000, 16, 700)])
def test_long_sums(rows, d, f):
    """Products with few tiles, whose K loops are split and joined."""
    check_backward(fp_module(), Block(rows, d, f, 5), "silu", "act8", dx_dtype=F32, dw_dtype=F32)


@pytest.mark.parametrize("rows,d,f,want", [(3000, 1000, 6000, (True, True)), (4999, 1001, 2500, (True, True)),
                                           (700, 2000, 1500, (True, True)), (3000, 1000, 6000, (True, False)),
                                           (3000, 1000, 6000, (False, True))])
def test_uneven_shares(rows, d, f, want):
    """Tiles of two lengths that come out in no whole rounds: some workers go ahead, the last tiles are in parts."""
    check_backward(fp_module(), Block(rows, d, f, rows), "silu", "none", want=want)


@pytest.mark.parametrize("want", [(True, False), (False, True), (False, False)])
def test_parts(want):
    check_backward(fp_module(), Block(100, 96, 200, 1), "gelu", "none", want=want)


def test_many_tiles():
    """More tiles than SMs in every product, so that blocks take several and their accumulators alternate."""
    fp = fp_module()
    b = Block(2600, 640, 2304, 9)
    check_forward(fp, b, "silu", "act8")
    check_backward(fp, b, "silu", "none")


def test_special_values():
    """NaN and infinities stay in the rows (and gradients) that the formulas put them in."""
    fp = fp_module()
    b = Block(200, 64, 160, 2)
    b.mx.t[3, 5] = float("nan")
    b.mx.t[150, 1] = float("inf")
    h = torch.empty(200, 160, dtype=BF16, device="cuda")
    gate, up = fp.Act8(200, 160), fp.Act8(200, 160)
    fp.fsdp_gated_ffn_forward(b.mx.t, b.mwg.t, b.mwu.t, h, gate=gate, up=up)
    bad = ~torch.isfinite(h).all(-1)
    assert bad.nonzero().flatten().tolist() == [3, 150] and bool(torch.isnan(h[3]).all())
    y = torch.empty_like(h)
    fp.fsdp_act8_load(gate, y)
    assert (~torch.isfinite(y).all(-1)).nonzero().flatten().tolist() == [3, 150]
    dx, dwg, dwu = torch.empty(200, 64, dtype=BF16, device="cuda"), torch.empty_like(b.mwg.t), torch.empty_like(b.mwu.t)
    fp.fsdp_gated_ffn_backward(b.mdh.t, b.mx.t, b.mwg.t, b.mwu.t, dx, dwg, dwu, gate=gate, up=up)
    assert (~torch.isfinite(dx).all(-1)).nonzero().flatten().tolist() == [3, 150]
    assert bool(torch.isnan(dwg).all())
    # Values far out on both sides: the activation's limits, no NaN.
    big = torch.tensor([[3e4] * 8, [-3e4] * 8], dtype=BF16, device="cuda")
    w = torch.ones(8, 8, dtype=BF16, device="cuda")
    for act, low in ((0, 0.0), (1, 0.0)):
        h = torch.empty(2, 8, dtype=BF16, device="cuda")
        fp.fsdp_gated_ffn_forward(big, w, w, h, activation=act)
        assert bool((h[0] > 5e10).all()) and bool((h[1] == low).all())


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gradient_against_differences(act):
    """Directional derivatives of sum(dh * h) with h in 64 bits.  dg and du are rounded to BF16 and each gradient to
    binary32 here, so a gradient's element is off by at most 2^-8 of its terms' magnitudes; over a direction of random
    signs that is at most 2^-8 of the sum of |v| times those magnitudes.  The central difference itself is good to 1e-7."""
    fp = fp_module()
    b = Block(40, 48, 72, 4)
    dx, dwg, dwu = (torch.empty(*s, device="cuda") for s in ((40, 48), (72, 48), (72, 48)))
    fp.fsdp_gated_ffn_backward(b.mdh.t, b.mx.t, b.mwg.t, b.mwu.t, dx, dwg, dwu, activation=ACTS[act])

    def loss(x, wg, wu):
        return float((b.dh * act_and_slope(x @ wg.T, act)[0] * (x @ wu.T)).sum())

    args = [b.x, b.wg, b.wu]
    g, u = b.x @ b.wg.T, b.x @ b.wu.T
    a, s = act_and_slope(g, act)
    mdg, mdu = (b.dh * u * s).abs(), (b.dh * a).abs()
    sizes = [mdg @ b.wg.abs() + mdu @ b.wu.abs(), mdg.T @ b.x.abs(), mdu.T @ b.x.abs()]
    step = 1e-5
    for k, grad in enumerate((dx, dwg, dwu)):
        v = normals(30 + k, *args[k].shape)
        hi, lo = [t.clone() for t in args], [t.clone() for t in args]
        hi[k] += step * v
        lo[k] -= step * v
        diff = (loss(*hi) - loss(*lo)) / (2 * step)
        got = float((grad.double().cpu() * v).sum())
        assert abs(got - diff) <= 2.0 ** -8 * 1.01 * float((sizes[k] * v.abs()).sum()) + 1e-6


def test_no_rows():
    fp = fp_module()
    x, h = torch.empty(0, 64, dtype=BF16, device="cuda"), torch.empty(0, 96, dtype=BF16, device="cuda")
    w = torch.ones(96, 64, dtype=BF16, device="cuda")
    fp.fsdp_gated_ffn_forward(x, w, w, h)
    m = [Matrix(96, 64, F32, 70) for _ in range(2)]
    fp.fsdp_gated_ffn_backward(h, x, w, w, x, m[0].t, m[1].t)
    assert all(bool((q.t == 0).all()) and q.intact() for q in m)


def test_same_bits_on_every_run_and_stream():
    fp = fp_module()
    b = Block(300, 200, 700, 8)
    side = torch.cuda.Stream()
    ws = torch.empty(fp.fsdp_gated_ffn_workspace(300, 200, 700, True), dtype=torch.uint8, device="cuda")
    outs = []
    for stream in (None, side, None):
        dx, dwg, dwu = (torch.empty(*s, device="cuda") for s in ((300, 200), (700, 200), (700, 200)))
        torch.cuda.synchronize()
        fp.fsdp_gated_ffn_backward(b.mdh.t, b.mx.t, b.mwg.t, b.mwu.t, dx, dwg, dwu, workspace=ws if stream is None else None,
                                   stream=stream)
        torch.cuda.synchronize()
        outs.append((dx, dwg, dwu))
    for o in outs[1:]:
        assert all(torch.equal(p, q) for p, q in zip(o, outs[0]))


@pytest.mark.parametrize("pad,offset", [(0, 1), (1, 0), (3, 5)])
def test_workspace_for_views(pad, offset):
    """A kept workspace of the size that the binding names is enough for views of aligned widths."""
    fp = fp_module()
    b = Block(140, 64, 96, 5, pad, offset)
    h, dx, dwg, dwu = (b.out(*s, BF16).t for s in ((140, 96), (140, 64), (96, 64), (96, 64)))
    ws = [torch.empty(fp.fsdp_gated_ffn_workspace(140, 64, 96, back, aligned=False), dtype=torch.uint8, device="cuda")
          for back in (False, True)]
    fp.fsdp_gated_ffn_forward(b.mx.t, b.mwg.t, b.mwu.t, h, workspace=ws[0])
    fp.fsdp_gated_ffn_backward(b.mdh.t, b.mx.t, b.mwg.t, b.mwu.t, dx, dwg, dwu, workspace=ws[1])
    want = [torch.empty(*s, dtype=BF16, device="cuda") for s in ((140, 96), (140, 64), (96, 64), (96, 64))]
    fp.fsdp_gated_ffn_forward(b.mx.t, b.mwg.t, b.mwu.t, want[0])
    fp.fsdp_gated_ffn_backward(b.mdh.t, b.mx.t, b.mwg.t, b.mwu.t, *want[1:])
    assert all(torch.equal(p, q) for p, q in zip((h, dx, dwg, dwu), want))


def test_workspace_comes_from_the_stream_of_the_call():
    """Scratch for a call on one stream is no block that another stream has just given back: what was launched there may
    still be at work on it.  (Memory only; nothing is launched.)"""
    fp_module()
    from fsdp2_gradient_packing_gb300 import fsdp_ops
    device, n, side = torch.cuda.current_device(), 1 << 22, torch.cuda.Stream()
    for current, other in ((torch.cuda.default_stream(), side), (side, torch.cuda.default_stream())):
        with torch.cuda.stream(current):
            given_back = torch.empty(n, dtype=torch.uint8, device="cuda").data_ptr()
            again = torch.empty(n, dtype=torch.uint8, device="cuda").data_ptr()
            assert again == given_back  # the allocator's own rule, within a stream
            at, size, _owner = fsdp_ops._workspace("here", None, n, other.cuda_stream, device)
            assert size == n and not given_back <= at < given_back + n
            at, size, _owner = fsdp_ops._workspace("here", None, n, current.cuda_stream, device)
            assert at == given_back
            assert torch.cuda.current_stream() == current


def test_in_a_graph():
    fp = fp_module()
    b = Block(140, 64, 96, 6)
    h, dx = torch.empty(140, 96, dtype=BF16, device="cuda"), torch.empty(140, 64, dtype=BF16, device="cuda")
    dwg, dwu = torch.empty(96, 64, device="cuda"), torch.empty(96, 64, device="cuda")
    gate, up = fp.Act8(140, 96), fp.Act8(140, 96)
    ws = torch.empty(fp.fsdp_gated_ffn_workspace(140, 64, 96, True), dtype=torch.uint8, device="cuda")

    def step():
        fp.fsdp_gated_ffn_forward(b.mx.t, b.mwg.t, b.mwu.t, h, gate=gate, up=up, workspace=ws)
        fp.fsdp_gated_ffn_backward(b.mdh.t, b.mx.t, b.mwg.t, b.mwu.t, dx, dwg, dwu, gate=gate, up=up, workspace=ws)

    step()
    torch.cuda.synchronize()
    want = [t.clone() for t in (h, dx, dwg, dwu)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t in (h, dx, dwg, dwu):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(want, (h, dx, dwg, dwu)))


def test_bounded_wait_reports():
    """A stage that is never filled: the waits give up, the status says so, and the next call is whole again."""
    fp = fp_module()
    b = Block(600, 640, 300, 7)
    h = torch.empty(600, 300, dtype=BF16, device="cuda")
    fp.fsdp_gated_ffn_forward(b.mx.t, b.mwg.t, b.mwu.t, h)
    fp.fsdp_ops_sync_status()
    fp.fsdp_debug_set_wait_fault(1, 20_000_000)
    try:
        fp.fsdp_gated_ffn_forward(b.mx.t, b.mwg.t, b.mwu.t, torch.empty_like(h))
        with pytest.raises(fp.FsdpError, match="gave up"):
            fp.fsdp_ops_sync_status()
    finally:
        fp.fsdp_debug_set_wait_fault(0, 0)
    again = torch.empty_like(h)
    fp.fsdp_gated_ffn_forward(b.mx.t, b.mwg.t, b.mwu.t, again)
    fp.fsdp_ops_sync_status()
    assert torch.equal(again, h)


def test_refusals():
    fp = fp_module()
    x, w = torch.zeros(4, 64, dtype=BF16, device="cuda"), torch.zeros(96, 64, dtype=BF16, device="cuda")
    h = torch.zeros(4, 96, dtype=BF16, device="cuda")
    with pytest.raises(ValueError, match="float32"):
        fp.fsdp_gated_ffn_forward(x.float(), w, w, h)
    with pytest.raises(ValueError, match="not 96 x 64"):
        fp.fsdp_gated_ffn_forward(x, w, w[:95], h)
    with pytest.raises(ValueError, match="together"):
        fp.fsdp_gated_ffn_forward(x, w, w, h, gate=h)
    with pytest.raises(ValueError, match="not an Act8"):
        fp.fsdp_gated_ffn_forward(x, w, w, h, gate=h, up=fp.Act8(4, 96))
    with pytest.raises(fp.FsdpError, match="unknown activation"):
        fp.fsdp_gated_ffn_forward(x, w, w, h, activation=7)
    with pytest.raises(ValueError, match="checkpoint of 4 x 64"):
        fp.fsdp_gated_ffn_forward(x, w, w, h, gate=fp.Act8(4, 64), up=fp.Act8(4, 96))
    with pytest.raises(ValueError, match="together"):
        fp.fsdp_gated_ffn_backward(h, x, w, w, x, w)
    with pytest.raises(ValueError, match="the call needs"):
        fp.fsdp_gated_ffn_backward(h, x, w, w, torch.empty_like(x), workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    # Straight through the C entry: an operand off a 16-byte boundary that the descriptor does not name.
    import ctypes
    d = fp.fsdp_ffn_desc_t(3, 64, 96, 64, 64, 64, 96, 96, 64, 64, 64, 0, 0, 1, 1, 1, 0)
    st = fp._lib.fsdp_gated_ffn_forward(ctypes.byref(d), x.data_ptr() + 2, w.data_ptr(), w.data_ptr(), h.data_ptr(), None, None,
                                        None, 0, None)
    assert st == fp.FSDP_EINVAL and "unaligned" in fp.fsdp_last_error()


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("rows", [1, 300])
def test_activation_over_its_range(act, rows):
    """g from -20 to 20 through unit weights (x and the identity), u = 1: h is act(g) to its own arithmetic and half an ulp,
    deep in the tail too; gradients of g likewise."""
    fp = fp_module()
    d = 64
    g = torch.linspace(-20, 20, rows * d).view(rows, d).to(BF16)
    x = torch.zeros(rows, d + 8, dtype=BF16)
    x[:, :d], x[:, d] = g, 1
    wg, wu = torch.zeros(d, d + 8, dtype=BF16), torch.zeros(d, d + 8, dtype=BF16)
    wg[:, :d], wu[:, d] = torch.eye(d), 1
    x, wg, wu = x.cuda(), wg.cuda(), wu.cuda()
    h, dh = torch.empty(rows, d, dtype=BF16, device="cuda"), torch.ones(rows, d, dtype=BF16, device="cuda")
    fp.fsdp_gated_ffn_forward(x, wg, wu, h, activation=ACTS[act])
    a, s = act_and_slope(g.double(), act)
    # The exponent's rounding grows with its argument, g or g^2 / 2: 2^-23 of it.
    fast = FAST + (g.double().abs() if act == "silu" else g.double().square() / 2) * 2.0 ** -23
    close(h, a, a.abs() * (fast + HALF[BF16]) + 1e-37, "h")
    dx = torch.empty(rows, d + 8, device="cuda")
    fp.fsdp_gated_ffn_backward(dh, x, wg, wu, dx, activation=ACTS[act])
    close(dx[:, :d], s, (1 + g.double().abs()) * fast + s.abs() * HALF[BF16] + 1e-37, "dx")

"""The gated linear recurrence, forward and backward, against its definition in 64 bits.

Tolerances, in units u = 2^-24, for a sequence of n rows.  a and 1 - a are off by at most 4 u each (an exponential of an
argument rounded once, whose slope times |z| stays below 1, a sum and a reciprocal), a step's two products and sum by 2 u more of
S, the largest magnitude among the sequence's inputs and its initial state, which bounds every state.  Errors shrink by a <= 1 a
step, so h is off by at most 10 (n + 1) u S, however the steps are grouped (a group's product of factors carries the same
roundings).  D is bounded by D+, the same recurrence over magnitudes, and off by at most 10 (n + 1) u D+.  1 - a alone is off by
(|z| + 6) u relative.  So dx is off by (1 - a) D+ (10 n + 20 + |z|) u, and dgate, with |h - x| <= 2 S, by a (1 - a) D+ S (30 n +
50 + 2 |z|) u; sums of dgate add a rounding of the sum of magnitudes a row."""
import threading

import numpy as np
import pytest
import torch

from gpu_util import fp_module
from ops_util import BF16, EPS32, F32, F64, HALF, Matrix, close, normals

pytestmark = pytest.mark.gpu
U = EPS32


def reference(x, z, initial, off, dh=None, dfinal=None):
    """Everything in 64 bits, row by row, with tolerances; off: where sequences begin and end.  Rows outside them are NaN."""
    x, z = x.double().numpy(), z.double().numpy()
    rows, cols = x.shape
    a, k = 1 / (1 + np.exp(-z)), 1 / (1 + np.exp(z))
    r = {n: np.full((rows, cols), np.nan) for n in ("h", "dx", "dz", "h_tol", "dx_tol", "dz_tol")}
    seqs = len(off) - 1
    h0 = np.zeros((seqs, cols)) if initial is None else initial.double().numpy()
    d0 = np.zeros((seqs, cols)) if dfinal is None else dfinal.double().numpy()
    r["final"], r["dinitial"], r["final_tol"], r["dinitial_tol"] = h0.copy(), d0.copy(), np.zeros((seqs, cols)), np.zeros((seqs, cols))
    for s in range(seqs):
        lo, hi = off[s], off[s + 1]
        n = hi - lo
        if n <= 0:
            continue
        top = np.maximum(np.abs(x[lo:hi]).max(0), np.abs(h0[s]))
        h = h0[s]
        for t in range(lo, hi):
            h = a[t] * h + k[t] * x[t]
            r["h"][t] = h
        r["h_tol"][lo:hi] = 10 * (n + 1) * U * top
        r["final"][s], r["final_tol"][s] = h, 10 * (n + 1) * U * top
        if dh is None:
            continue
        d, plus = d0[s], np.abs(d0[s])
        g = dh.double().numpy()
        for t in range(hi - 1, lo - 1, -1):
            d, plus = d + g[t], plus + np.abs(g[t])
            before = r["h"][t - 1] if t > lo else h0[s]
            r["dx"][t], r["dz"][t] = k[t] * d, d * (before - x[t]) * a[t] * k[t]
            r["dx_tol"][t] = k[t] * plus * (10 * n + 20 + np.abs(z[t])) * U
            r["dz_tol"][t] = a[t] * k[t] * plus * top * (30 * n + 50 + 2 * np.abs(z[t])) * U
            d, plus = d * a[t], plus * a[t]
        r["dinitial"][s], r["dinitial_tol"][s] = d, (10 * n + 20) * U * plus
    return {n: torch.from_numpy(v) for n, v in r.items()}


def near(got, want, tol, dtype, what):
    close(got, want, tol + (want.abs() + tol) * HALF[dtype] + 1e-38, what)


def check(fp, rows, cols, lengths=None, off=None, dtype=F32, h_dtype=None, dx_dtype=None, bias="f32", with_states=True, ld=None, offset=0,
          seed=0, index=torch.int64, backward=True, slow=4.0):
    """lengths: rows of every sequence (one call with seq_len); off: packed sequences."""
    h_dtype, dx_dtype = h_dtype or dtype, dx_dtype or dtype
    x, gate = normals(seed, rows, cols).to(dtype), normals(seed + 1, rows, cols, std=1.5).to(dtype)
    b = None if bias is None else (slow * torch.rand(cols, generator=torch.Generator().manual_seed(seed), dtype=F64)).to(BF16 if bias == "bf16" else F32)
    z = gate.double() + (0 if b is None else b.double())
    where = dict(seq_len=lengths) if off is None else dict(offsets=torch.tensor(off).to(index).cuda())
    off = off if off is not None else [k * lengths for k in range(rows // lengths + 1)]
    seqs = len(off) - 1
    initial, dfinal = (normals(seed + 2 + k, seqs, cols).float() if with_states else None for k in range(2))
    dh = normals(seed + 4, rows, cols).to(h_dtype)
    want = reference(x, z, initial, off, dh, dfinal)
    mx, mg = Matrix(rows, cols, dtype, ld, offset, x), Matrix(rows, cols, dtype, ld, offset, gate)
    mh, mdh = Matrix(rows, cols, h_dtype, ld, offset), Matrix(rows, cols, h_dtype, ld, offset, dh)
    dev = [None if t is None else t.cuda() for t in (b, initial, dfinal)]
    final = torch.full((seqs, cols), 9.0, device="cuda") if with_states else None
    states = torch.full((fp.fsdp_gated_scan_states(rows, cols), cols), float("nan"), device="cuda")
    covered = torch.zeros(rows, dtype=torch.bool)
    for s in range(seqs):
        covered[off[s]:off[s + 1]] = True
    untouched = mh.t.clone()
    fp.fsdp_gated_scan_forward(mx.t, mg.t, mh.t, bias=dev[0], initial=dev[1], final=final, states=states if backward else None, **where)
    near(mh.t[covered.cuda()], want["h"][covered], want["h_tol"][covered], h_dtype, "h")
    assert torch.equal(mh.t[~covered.cuda()].view(torch.uint8), untouched[~covered.cuda()].view(torch.uint8))
    if with_states:
        near(final, want["final"], want["final_tol"], F32, "final")
    assert mh.intact() and mx.intact() and mg.intact()
    if not backward:
        return
    mdx, mdg = Matrix(rows, cols, dx_dtype, ld, offset), Matrix(rows, cols, dx_dtype, ld, offset)
    untouched = mdx.t.clone()
    dinitial = torch.full((seqs, cols), 9.0, device="cuda") if with_states else None
    dbias = None if b is None else torch.full_like(dev[0], 9.0)
    fp.fsdp_gated_scan_backward(mdh.t, mx.t, mg.t, states, mdx.t, mdg.t, bias=dev[0], dbias=dbias, initial=dev[1], dinitial=dinitial,
                                dfinal=dev[2], **where)
    near(mdx.t[covered.cuda()], want["dx"][covered], want["dx_tol"][covered], dx_dtype, "dx")
    near(mdg.t[covered.cuda()], want["dz"][covered], want["dz_tol"][covered], dx_dtype, "dgate")
    for m in (mdx, mdg):
        assert torch.equal(m.t[~covered.cuda()].view(torch.uint8), untouched[~covered.cuda()].view(torch.uint8)) and m.intact()
    if with_states:
        near(dinitial, want["dinitial"], want["dinitial_tol"], F32, "dinitial")
    if dbias is not None:
        dz = want["dz"][covered]
        near(dbias, dz.sum(0), want["dz_tol"][covered].sum(0) + (rows + 16) * U * dz.abs().sum(0), b.dtype, "dbias")


KINDS = [dict(), dict(dtype=BF16), dict(dtype=BF16, h_dtype=F32, dx_dtype=F32, bias="bf16"), dict(h_dtype=BF16, dx_dtype=BF16, bias=None)]


@pytest.mark.parametrize("kind", range(len(KINDS)))
@pytest.mark.parametrize("cols", [1, 2, 31, 32, 33, 64, 66, 129, 200, 515])
def test_widths(cols, kind):
    check(fp_module(), 300, cols, 150, seed=cols, **KINDS[kind])


@pytest.mark.parametrize("length", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 257, 1000])
@pytest.mark.parametrize("seqs", [1, 3])
def test_lengths(length, seqs):
    check(fp_module(), length * seqs, 70, length, seed=length, dtype=BF16)
    check(fp_module(), length * seqs, 68, length, seed=length, with_states=False)


def test_one_long_sequence():
    """More tiles than fit the device at once would have to wait for one another: the carries pass from tile to tile."""
    check(fp_module(), 20011, 70, 20011, dtype=BF16, slow=8.0)


@pytest.mark.parametrize("off", [[0, 0], [0, 300], [0, 0, 0, 5, 5, 130, 131, 259, 300, 300], [0, 128, 256, 300], [0, 100, 250], [7, 50, 290],
                                 [300, 300], [50, 50, 60], [0, 1, 2, 3, 4, 299]])
@pytest.mark.parametrize("index", [torch.int32, torch.int64])
def test_packed(off, index):
    """Empty sequences, borders inside and between tiles, rows before the first and behind the last sequence."""
    check(fp_module(), 300, 70, off=off, index=index, seed=len(off))
    check(fp_module(), 300, 64, off=off, index=index, dtype=BF16, with_states=False)


def test_packed_at_random():
    rng = np.random.default_rng(5)
    for seed in range(6):
        rows = int(rng.integers(1, 1500))
        off = [0] + sorted(int(v) for v in rng.integers(0, rows + 1, int(rng.integers(0, 40)))) + [rows]
        check(fp_module(), rows, int(rng.integers(1, 150)), off=off, seed=seed, dtype=BF16 if seed % 2 else F32)


@pytest.mark.parametrize("ld,offset", [(64, 1), (72, 0), (65, 0), (64, 8), (66, 2)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_strides(ld, offset, dtype):
    check(fp_module(), 200, 64, 100, dtype=dtype, ld=ld, offset=offset)


def test_no_rows():
    fp = fp_module()
    e = torch.empty(0, 64, device="cuda")
    initial, final, dbias = torch.randn(3, 64, device="cuda"), torch.empty(3, 64, device="cuda"), torch.full((64,), 9.0, device="cuda")
    off = torch.zeros(4, dtype=torch.int64, device="cuda")
    fp.fsdp_gated_scan_forward(e, e, e, initial=initial, final=final, offsets=off)
    assert torch.equal(initial, final)
    fp.fsdp_gated_scan_backward(e, e, e, e, e, e, bias=torch.zeros(64, device="cuda"), dbias=dbias, dinitial=final, dfinal=initial * 2, offsets=off)
    assert bool((dbias == 0).all()) and torch.equal(final, initial * 2)
    fp.fsdp_gated_scan_forward(e, e, e, seq_len=5)


def test_generation_in_place_continues_a_sequence():
    """Rows one at a time, the state in one buffer, and pieces of a sequence give what the whole gives."""
    fp = fp_module()
    x, gate, bias = (torch.randn(*s, device="cuda") for s in ((40, 96), (40, 96), (96,)))
    whole, state = torch.empty_like(x), torch.zeros(1, 96, device="cuda")
    fp.fsdp_gated_scan_forward(x, gate, whole, bias=bias, seq_len=40)
    h = torch.empty_like(x)
    for t in range(40):
        fp.fsdp_gated_scan_forward(x[t:t + 1], gate[t:t + 1], h[t:t + 1], bias=bias, initial=state, final=state, seq_len=1)
    close(h, whole, 10 * 41 * 2 * U * float(x.abs().max()), "h")
    close(state, whole[-1:], 10 * 41 * 2 * U * float(x.abs().max()), "state")
    # A state of many sequences, updated in place over several rows.
    state = torch.randn(8, 96, device="cuda")
    apart = torch.empty_like(state)
    fp.fsdp_gated_scan_forward(x, gate, h, initial=state, final=apart, seq_len=5)
    fp.fsdp_gated_scan_forward(x, gate, h, initial=state, final=state, seq_len=5)
    assert torch.equal(state, apart)
    # A sequence that fills many tiles, in place.
    xl, gl = (torch.randn(3000, 96, device="cuda") for _ in range(2))
    hl, state = torch.empty_like(xl), torch.randn(1, 96, device="cuda")
    apart = torch.empty_like(state)
    fp.fsdp_gated_scan_forward(xl, gl + 6, hl, initial=state, final=apart, seq_len=3000)
    fp.fsdp_gated_scan_forward(xl, gl + 6, hl, initial=state, final=state, seq_len=3000)
    assert torch.equal(state, apart)


def test_extreme_gates():
    """Gates far out: the state is kept or replaced exactly; infinite ones too; a NaN stays in its column and behind its row."""
    fp = fp_module()
    x = torch.randn(300, 64, device="cuda")
    for value, kept in ((200.0, True), (float("inf"), True), (-200.0, False), (-float("inf"), False)):
        gate, initial, h = torch.full_like(x, value), torch.randn(1, 64, device="cuda"), torch.empty_like(x)
        states = torch.empty(fp.fsdp_gated_scan_states(300, 64), 64, device="cuda")
        fp.fsdp_gated_scan_forward(x, gate, h, initial=initial, seq_len=300, states=states)
        assert torch.equal(h, initial.expand(300, 64) if kept else x)
        dx, dgate, dinitial = torch.empty_like(x), torch.empty_like(x), torch.empty_like(initial)
        fp.fsdp_gated_scan_backward(torch.ones_like(x), x, gate, states, dx, dgate, initial=initial, dinitial=dinitial, seq_len=300)
        assert bool((dgate == 0).all()) and bool((dx == (0.0 if kept else 1.0)).all()) and bool((dinitial == (300.0 if kept else 0.0)).all())
    gate = torch.zeros_like(x)
    x[140, 5] = float("nan")
    fp.fsdp_gated_scan_forward(x, gate, h, seq_len=150)
    assert bool(torch.isnan(h[140:150, 5]).all())
    h[140:150, 5] = 0.0
    assert bool(torch.isfinite(h).all())


def test_gradients_against_differences():
    """Central differences of <dh, h> + <dfinal, final> along random directions, in 32 bits: the step of 2^-6 leaves a third-order
    term below 2e-4 of the inner product's scale and 1e-4 from the outputs' rounding."""
    fp = fp_module()
    rows, cols = 90, 40
    gen = torch.Generator(device="cuda").manual_seed(3)
    x, gate, bias, h0, dh, df = (torch.randn(*s, generator=gen, device="cuda") for s in ((rows, cols), (rows, cols), (cols,), (3, cols),
                                                                                        (rows, cols), (3, cols)))
    v = [torch.randn(t.shape, generator=gen, device="cuda") for t in (x, gate, bias, h0)]

    def value(e):
        h, final = torch.empty_like(x), torch.empty_like(h0)
        fp.fsdp_gated_scan_forward(x + e * v[0], gate + e * v[1], h, bias=bias + e * v[2], initial=h0 + e * v[3], final=final, seq_len=30)
        return float((h.double() * dh.double()).sum() + (final.double() * df.double()).sum())

    states, h = torch.empty(fp.fsdp_gated_scan_states(rows, cols), cols, device="cuda"), torch.empty_like(x)
    fp.fsdp_gated_scan_forward(x, gate, h, bias=bias, initial=h0, seq_len=30, states=states)
    g = [torch.empty_like(t) for t in (x, gate, bias, h0)]
    fp.fsdp_gated_scan_backward(dh, x, gate, states, g[0], g[1], bias=bias, dbias=g[2], initial=h0, dinitial=g[3], dfinal=df, seq_len=30)
    want = sum(float((a.double() * b.double()).sum()) for a, b in zip(g, v))
    got = (value(2.0 ** -6) - value(-2.0 ** -6)) * 2.0 ** 5
    scale = sum(float((a.double() * b.double()).abs().sum()) for a, b in zip(g, v))
    assert abs(got - want) <= 3e-4 * scale


def test_same_bits_streams_graphs_and_threads():
    fp = fp_module()
    rows, cols = 20000, 200
    x, gate, dh = (torch.randn(rows, cols, device="cuda").to(BF16) for _ in range(3))
    bias = torch.rand(cols, device="cuda") * 6
    off = torch.tensor([0, 700, 700, 15001, rows], device="cuda")
    n = fp.fsdp_gated_scan_states(rows, cols)

    def outputs():
        return [torch.zeros(n, cols, device="cuda")] + [torch.empty_like(x) for _ in range(3)] + [torch.empty_like(bias)]

    def go(out, workspaces=(None, None), stream=None):
        states, h, dx, dgate, dbias = out
        fp.fsdp_gated_scan_forward(x, gate, h, bias=bias, states=states, offsets=off, workspace=workspaces[0], stream=stream)
        fp.fsdp_gated_scan_backward(dh, x, gate, states, dx, dgate, bias=bias, dbias=dbias, offsets=off, workspace=workspaces[1], stream=stream)

    first, again = outputs(), outputs()
    go(first)
    for _ in range(5):
        go(again)
        assert all(torch.equal(a, b) for a, b in zip(first[1:], again[1:]))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = outputs()
    side.wait_stream(torch.cuda.current_stream())
    go(again, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first[1:], again[1:]))
    # Two captured calls that share their workspaces, replayed in turn after the workspace held something else.
    ws = [torch.empty(max(1, fp.fsdp_gated_scan_workspace(rows, cols, 4, True, k)), dtype=torch.uint8, device="cuda") for k in (False, True)]
    held = [outputs(), outputs()]
    graphs = []
    for k in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[k]):
            go(held[k], ws)
    for k in (0, 1, 0):
        for t in held[k] + ws:
            t.fill_(7)
        graphs[k].replay()
        assert all(torch.equal(a, b) for a, b in zip(first[1:], held[k][1:]))
    got = [outputs(), outputs()]
    torch.cuda.synchronize()

    def many(k):
        s = torch.cuda.Stream()
        for _ in range(10):
            go(got[k], stream=s)
        s.synchronize()

    threads = [threading.Thread(target=many, args=(k,)) for k in range(2)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    for k in range(2):
        assert all(torch.equal(a, b) for a, b in zip(first[1:], got[k][1:]))
    fp.fsdp_ops_sync_status()


def test_offsets_that_break_the_rules_touch_nothing_else():
    """Decreasing offsets, and offsets far outside the rows: results are unspecified, memory beside the arrays is not."""
    fp = fp_module()
    for off in ([0, 200, 100, 300], [300, 0], [-5, 10_000_000], [1 << 40, -(1 << 40), 50], [100, 100, 0, 0, 300]):
        seqs = len(off) - 1
        mx, mg, mh, mdx, mdg = (Matrix(300, 70, F32, value=torch.randn(300, 70)) for _ in range(5))
        mi, mf = Matrix(seqs, 70, F32, value=torch.randn(seqs, 70)), Matrix(seqs, 70, F32)
        ms = Matrix(fp.fsdp_gated_scan_states(300, 70), 70, F32, value=0.0)
        o = torch.tensor(off, device="cuda")
        fp.fsdp_gated_scan_forward(mx.t, mg.t, mh.t, initial=mi.t, final=mf.t, states=ms.t, offsets=o)
        fp.fsdp_gated_scan_backward(mh.t, mx.t, mg.t, ms.t, mdx.t, mdg.t, initial=mi.t, dinitial=mf.t, offsets=o)
        fp.fsdp_ops_sync_status()
        assert all(m.intact() for m in (mx, mg, mh, mdx, mdg, mi, mf, ms))


def test_binding_refusals():
    fp = fp_module()
    x = torch.empty(12, 16, device="cuda")
    ok = dict(seq_len=4)
    s = torch.empty(3, 16, device="cuda")
    bad = [((x, x.to(BF16), x), ok, "different dtypes"), ((x, x, x), {}, "either"), ((x, x, x), dict(seq_len=5), "not sequences"),
           ((x, x, x), dict(seq_len=4, offsets=torch.zeros(2, dtype=torch.int64, device="cuda")), "either"),
           ((x, x, x), dict(offsets=torch.zeros(0, dtype=torch.int64, device="cuda")), "empty"),
           ((x, x, x), dict(offsets=torch.zeros(2, device="cuda")), "not one of"), ((x, x, x), dict(seq_len=4, initial=s[:2]), "not 3"),
           ((x, x, x), dict(seq_len=4, final=s.to(BF16)), "bfloat16"), ((x, x, x), dict(seq_len=4, bias=s), "vector"),
           ((x, x, x), dict(seq_len=4, initial=torch.empty(3, 20, device="cuda")[:, :16]), "gaps"),
           ((x, x, x), dict(seq_len=4, states=torch.empty(9, 16, device="cuda")), "states")]
    for args, kw, word in bad:
        with pytest.raises(ValueError, match=word):
            fp.fsdp_gated_scan_forward(*args, **kw)
    with pytest.raises(ValueError, match="states is needed"):
        fp.fsdp_gated_scan_backward(x, x, x, None, x, x, seq_len=4)


@pytest.mark.parametrize("kind", range(len(KINDS)))
@pytest.mark.parametrize("rows,cols,ld,offset", [(1, 1, None, 0), (1, 4096, None, 0), (70, 130, None, 0), (5, 515, None, 0), (200, 64, 65, 1), (3, 128, 130, 2)])
def test_one_row_sequences(rows, cols, ld, offset, kind):
    """Steps of generation, aligned and not, through the backward pass too."""
    check(fp_module(), rows, cols, 1, ld=ld, offset=offset, seed=rows + cols, **KINDS[kind])
    check(fp_module(), rows, cols, 1, ld=ld, offset=offset, seed=rows + cols, with_states=False, **KINDS[kind])


@pytest.mark.parametrize("seqs,length,cols,dtype", [(3, 1536, 70, BF16), (3, 1536, 64, F32), (2, 2560, 200, BF16), (5, 128, 66, BF16),
                                                    (9, 640, 1100, BF16)])
def test_sequences_of_whole_tiles(seqs, length, cols, dtype):
    """Sequences that begin where tiles do, many tiles long: they are gone through side by side."""
    check(fp_module(), seqs * length, cols, length, dtype=dtype, seed=length, slow=7.0)

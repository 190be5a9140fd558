"""The gated linear recurrence where 1 - a or a is small: slow columns that begin from no state, states that decay at once, gradients
that come through rows without one.  Every element against its own size, not that of the inputs.

Tolerances, in units u = 2^-24.  e = 2^(-z log2 e): z is a rounded sum (|z| u), its product with a rounded constant 2 |z| u more, the
exponential 2 ulp, so e is off by (3 |z| + 4) u relative.  a = 1 / (1 + e) takes (1 - a) of that, and 3 u for a sum and a
reciprocal (and at most 2^-125, where gates are as good as shut); 1 - a = e a takes a of it, and 4 u.  With H+ the recurrence over magnitudes, a row's error is a times the
error before it, a H+ times what a is off by, (1 - a) |x| times what 1 - a is off by, and a few u of H+ for products, sums and the
factors of whole groups of rows (1 - K with K the recurrence of ones, at K < 1/2, which doubles the factor's share of e's error).
D goes the same way from the last row to the first."""
import numpy as np
import pytest
import torch

from gpu_util import fp_module
from ops_util import BF16, EPS32, F32, F64, HALF, Matrix, close, normals

pytestmark = pytest.mark.gpu
U = EPS32
TINY = 1e-37  # results below the least normal number


def gates(z):
    a, k = 1 / (1 + np.exp(-z)), 1 / (1 + np.exp(z))
    e = (6 * np.abs(z) + 8) * U
    return a, k, k * e + 3 * U + 2.0 ** -125 / a, a * e + 4 * U


def states(x, z, h0):
    """(h, its tolerance), with row 0 the initial state."""
    a, k, da, dk = gates(z)
    h, plus, tol = [h0], [np.abs(h0)], [np.zeros_like(h0)]
    for t in range(len(x)):
        plus.append(a[t] * plus[-1] + k[t] * np.abs(x[t]))
        tol.append(a[t] * (tol[-1] + (da[t] + 2 * U) * plus[-2]) + k[t] * np.abs(x[t]) * (dk[t] + 3 * U) + 3 * U * plus[-1])
        h.append(a[t] * h[-1] + k[t] * x[t])
    return np.stack(h), np.stack(tol)


def gradients(x, z, h, h_tol, dh, dfinal):
    a, k, da, dk = gates(z)
    d, plus, tol = dfinal, np.abs(dfinal), np.zeros_like(dfinal)
    out = {n: np.zeros_like(x) for n in ("dx", "dx_tol", "dz", "dz_tol")}
    for t in range(len(x) - 1, -1, -1):
        d, plus = d + dh[t], plus + np.abs(dh[t])
        tol = tol + 3 * U * plus
        gap = np.abs(h[t] - x[t])
        gap_tol = h_tol[t] + 2 * U * (np.abs(h[t]) + np.abs(x[t]))
        out["dx"][t], out["dx_tol"][t] = k[t] * d, k[t] * (tol + plus * (dk[t] + 2 * U))
        out["dz"][t] = d * (h[t] - x[t]) * a[t] * k[t]
        out["dz_tol"][t] = a[t] * k[t] * (tol * (gap + gap_tol) + plus * (gap_tol + gap * (da[t] + dk[t] + 5 * U)))
        tol = a[t] * (tol + plus * (da[t] + 2 * U))
        d, plus = a[t] * d, a[t] * plus
    return dict(out, dinitial=d, dinitial_tol=tol + 2 * U * plus)


def near(got, want, tol, what):
    want, tol = (torch.from_numpy(v) for v in (want, tol))
    close(got, want, tol + (want.abs() + tol) * HALF[got.dtype] + TINY, what)


def layer(rows, cols, low, high, dtype, seed):
    """x, gate and bias: columns whose gates lie around low .. high."""
    bias = torch.linspace(low, high, cols, dtype=F64).float()
    return normals(seed, rows, cols).to(dtype), normals(seed + 1, rows, cols, std=0.25).to(dtype), bias


def check(rows, cols, length, low, high, dtype=F32, h_dtype=F32, seed=0, x=None, initial=None, dh=None, dfinal=None):
    """Forward and backward over sequences of one length; x, dh: changes to what normals gave."""
    fp = fp_module()
    xs, gate, bias = layer(rows, cols, low, high, dtype, seed)
    xs = xs if x is None else x(xs)
    grads = normals(seed + 2, rows, cols).to(h_dtype)
    grads = grads if dh is None else dh(grads)
    z = gate.double().numpy() + bias.double().numpy()
    seqs = rows // length
    states_out = torch.full((fp.fsdp_gated_scan_states(rows, cols), cols), float("nan"), device="cuda")
    h, final = Matrix(rows, cols, h_dtype), torch.empty(seqs, cols, device="cuda")
    dev = [None if t is None else t.cuda() for t in (initial, dfinal)]
    fp.fsdp_gated_scan_forward(xs.cuda(), gate.cuda(), h.t, bias=bias.cuda(), initial=dev[0], final=final, states=states_out, seq_len=length)
    dx, dgate = (torch.empty(rows, cols, dtype=dtype, device="cuda") for _ in range(2))
    dinitial = torch.empty(seqs, cols, device="cuda")
    fp.fsdp_gated_scan_backward(grads.cuda(), xs.cuda(), gate.cuda(), states_out, dx, dgate, bias=bias.cuda(), initial=dev[0], dinitial=dinitial,
                                dfinal=dev[1], seq_len=length)
    none = np.zeros(cols)
    for s in range(seqs):
        at = slice(s * length, (s + 1) * length)
        xn, zn, gn = xs[at].double().numpy(), z[at], grads[at].double().numpy()
        want, tol = states(xn, zn, none if initial is None else initial[s].double().numpy())
        near(h.t[at], want[1:], tol[1:], f"h of sequence {s}")
        near(final[s], want[-1], tol[-1], f"final of sequence {s}")
        g = gradients(xn, zn, want, tol, gn, none if dfinal is None else dfinal[s].double().numpy())
        near(dx[at], g["dx"], g["dx_tol"], f"dx of sequence {s}")
        near(dgate[at], g["dz"], g["dz_tol"], f"dgate of sequence {s}")
        near(dinitial[s], g["dinitial"], g["dinitial_tol"], f"dinitial of sequence {s}")
    assert h.intact()


@pytest.mark.parametrize("cols", [64, 70])
@pytest.mark.parametrize("length", [2, 5, 16, 40, 300, 2100])
def test_slow_columns_from_no_state(length, cols):
    """h is far smaller than x: it has the precision of 1 - a, not that of a."""
    check(length * (1 if length > 1000 else 3), cols, length, 6.0, 16.0, seed=length)


@pytest.mark.parametrize("cols", [64, 70])
def test_slow_columns_in_bf16(cols):
    """Inputs in BF16 with h and its gradient in FP32, and all in BF16."""
    check(600, cols, 300, 6.0, 16.0, dtype=BF16, seed=1)
    check(600, cols, 300, 6.0, 16.0, dtype=BF16, h_dtype=BF16, seed=2)


@pytest.mark.parametrize("call", [1, 2, 3, 16])
def test_a_sequence_cut_into_calls(call):
    """States handed from call to call: the same tokens, however they are cut."""
    fp = fp_module()
    rows, cols = 1536, 66
    x, gate, bias = layer(rows, cols, 6.0, 16.0, F32, call)
    state = torch.zeros(1, cols, device="cuda")
    h = torch.empty(rows, cols, device="cuda")
    xs, gs, b = x.cuda(), gate.cuda(), bias.cuda()
    for t in range(0, rows, call):
        at = slice(t, t + call)
        fp.fsdp_gated_scan_forward(xs[at], gs[at], h[at], bias=b, initial=state, final=state, seq_len=call)
    want, tol = states(x.double().numpy(), gate.double().numpy() + bias.double().numpy(), np.zeros(cols))
    near(h, want[1:], tol[1:], "h")
    near(state[0], want[-1], tol[-1], "final")


@pytest.mark.parametrize("cols", [64, 70])
@pytest.mark.parametrize("length", [3, 16, 150])
def test_states_that_decay_at_once(length, cols):
    """Rows without input behind a large state: h has the precision of a, not that of 1 - a."""
    seqs = 3
    initial = normals(7, seqs, cols, std=1e6).float()
    check(length * seqs, cols, length, -14.0, -2.0, seed=length, initial=initial, x=torch.zeros_like)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("cols", [64, 70])
@pytest.mark.parametrize("length", [3, 16, 150])
def test_gradients_through_rows_without_one(length, cols, dtype):
    """dh is 0 at all rows but every seventh: D between them is a D and nothing else."""
    rows = length * 3
    kept = (torch.arange(rows) % 7 == 2)[:, None]
    check(rows, cols, length, -14.0, 2.0, dtype=dtype, h_dtype=dtype, seed=length, dh=lambda g: torch.where(kept, g, torch.zeros_like(g)),
          initial=normals(8, 3, cols).float(), dfinal=normals(9, 3, cols).float())


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_gates_that_are_shut_or_open(dtype):
    """Gates of +-infinity and +-1e4: a is 0 or 1, and every result is what the formulas say."""
    fp = fp_module()
    rows, cols = 40, 70
    x, gate = normals(3, rows, cols).to(dtype), normals(4, rows, cols).to(dtype)
    gate[5], gate[11], gate[17], gate[23] = float("-inf"), float("inf"), -1e4, 1e4
    a = torch.sigmoid(gate.double())
    h, want = torch.empty(rows, cols, device="cuda"), []
    fp.fsdp_gated_scan_forward(x.cuda(), gate.cuda(), h, seq_len=rows)
    state = torch.zeros(cols, dtype=F64)
    for t in range(rows):
        state = a[t] * state + (1 - a[t]) * x[t].double()
        want.append(state)
    close(h, torch.stack(want), 10 * (rows + 1) * U * float(x.double().abs().max()), "h")
    for t in (5, 17):
        assert torch.equal(h[t].cpu(), x[t].float())
    for t in (11, 23):
        assert torch.equal(h[t], h[t - 1])


@pytest.mark.parametrize("cols", [64, 70])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_gates_that_are_nearly_shut(dtype, cols):
    """From where odds are large to where they leave the range of binary32, in some columns and rows of a tile and not in others."""
    initial = normals(10, 3, cols).float()
    check(450, cols, 150, -130.0, -30.0, dtype=dtype, h_dtype=dtype, seed=5, initial=initial)
    check(450, cols, 150, -75.0, -65.0, dtype=dtype, h_dtype=dtype, seed=6, initial=initial)
    check(450, cols, 150, -100.0, 40.0, dtype=dtype, h_dtype=dtype, seed=7, initial=initial)


@pytest.mark.parametrize("cols", [64, 70])
def test_large_inputs_at_shut_gates(cols):
    """Odds times inputs beyond the range of binary32, where every result lies within it."""
    check(300, cols, 150, -60.0, 10.0, seed=8, x=lambda v: v * 1e30, initial=normals(11, 2, cols, std=1e30).float())


def test_resets():
    """Rows of x = 0 at a gate of -infinity, here and there: the state is 0 from there on, exactly, over rows, warps and tiles."""
    fp = fp_module()
    rows, cols = 400, 70
    x, gate = torch.zeros(rows, cols), normals(12, rows, cols).float()
    reset = 37
    gate[reset] = float("-inf")
    h, final = torch.empty(rows, cols, device="cuda"), torch.empty(1, cols, device="cuda")
    initial = torch.ones(1, cols, device="cuda") * 1e30
    states = torch.empty(fp.fsdp_gated_scan_states(rows, cols), cols, device="cuda")
    fp.fsdp_gated_scan_forward(x.cuda(), gate.cuda(), h, initial=initial, final=final, states=states, seq_len=rows)
    assert bool((h[:5] > 0).all()) and bool((h[reset:] == 0).all()) and bool((final == 0).all())
    dx, dgate, dinitial = torch.empty_like(h), torch.empty_like(h), torch.empty_like(final)
    dh = torch.zeros(rows, cols)
    dh[300] = 1e30
    fp.fsdp_gated_scan_backward(dh.cuda(), x.cuda(), gate.cuda(), states, dx, dgate, initial=initial, dinitial=dinitial, seq_len=rows)
    assert bool((dx[:reset] == 0).all()) and bool((dgate[:reset + 1] == 0).all()) and bool((dinitial == 0).all())


@pytest.mark.parametrize("dtype,cols", [(F32, 64), (F32, 67), (BF16, 64), (BF16, 67)])
@pytest.mark.parametrize("with_initial", [False, True])
def test_states_of_sequences_of_one_row(dtype, cols, with_initial):
    """A forward call fills the states for the backward call, whatever the sequences' length."""
    fp = fp_module()
    rows = 300
    x, gate = normals(13, rows, cols).to(dtype).cuda(), normals(14, rows, cols).to(dtype).cuda()
    initial = normals(15, rows, cols).float().cuda() if with_initial else None
    states = torch.full((fp.fsdp_gated_scan_states(rows, cols), cols), float("nan"), device="cuda")
    h = torch.empty_like(x)
    fp.fsdp_gated_scan_forward(x, gate, h, initial=initial, seq_len=1, states=states)
    assert torch.equal(states, torch.zeros_like(states) if initial is None else initial[::64])
    dh, dx, dgate, dinitial = torch.ones_like(x), torch.empty_like(x), torch.empty_like(x), torch.empty(rows, cols, device="cuda")
    fp.fsdp_gated_scan_backward(dh, x, gate, states, dx, dgate, initial=initial, dinitial=dinitial, seq_len=1)
    assert all(bool(torch.isfinite(t).all()) for t in (dx, dgate, dinitial))


@pytest.mark.parametrize("cols", [64, 70])
def test_states_near_the_end_of_the_range(cols):
    """A state and inputs whose sum leaves the range of binary32, and whose mean does not."""
    initial = torch.full((2, cols), 3.3e38)
    check(300, cols, 150, -1.0, 1.0, seed=16, x=lambda v: (0.5 + 0.5 * torch.sigmoid(v)) * 1e38, initial=initial)
    check(300, cols, 150, 3.0, 9.0, seed=17, x=lambda v: (0.5 + 0.5 * torch.sigmoid(v)) * 1e38, initial=-initial)
    check(300, cols, 150, 2.0, 4.0, seed=18, x=lambda v: (0.99 + 0.01 * torch.sigmoid(v)) * 3.3e38, initial=initial)

"""Distillation and clipped policy losses, values and gradients, against their definitions in 64 bits.

Tolerances, in units u = 2^-24.  With Z the largest |z / T| of a row plus 1: a scaled logit minus the row's maximum, times log2 e, is
off by at most 8 u Z, an exponential by that and 4 u relative, their sum by 256 u more (chains of at most 256 additions), so lse is off
by d = (8 Z + 270 + 2 |lse|) u, and a probability by d + (8 Z + 8) u relative.  The teacher's entries count the same way with their own
largest magnitude.  What a formula makes of these is their sum over its terms; a result in a narrower type adds half an ulp of it."""
import math
import threading

import pytest
import torch

from gpu_util import fp_module
from ops_util import BF16, EPS32, F32, F64, HALF, Matrix, close, normals

pytestmark = pytest.mark.gpu
U = EPS32
INF = float("inf")


def softmax_parts(logits, t):
    """(scaled logits, lse, p, tolerance of lse, relative tolerance of p) in 64 bits."""
    z = logits.double() / t
    lse = torch.logsumexp(z, -1)
    big = torch.where(torch.isfinite(z), z.abs(), 0.0).amax(-1) + 1
    d = (8 * big + 270 + 2 * lse.abs()) * U
    return z, lse, torch.exp(z - lse[:, None]), d, (d + (8 * big + 8) * U)[:, None]


def teacher_parts(ids, teacher, vocab, t):
    """(entries that count, q, log q, relative tolerance of q) in 64 bits."""
    v = teacher.double() / t
    here = (ids >= 0) & (ids < vocab) & (v > -INF)
    v = torch.where(here, v, -INF)
    lse = torch.logsumexp(v, -1, keepdim=True)
    log_q = torch.where(here, v - lse, 0.0)
    q = torch.where(here, torch.exp(log_q), 0.0)
    big = torch.where(here, v.abs(), 0.0).amax(-1, keepdim=True) + 1
    return here, q, log_q, (20 * big + 300) * U


def distill_reference(logits, ids, teacher, t, w, dloss):
    rows, vocab = logits.shape
    z, lse, p, d, rel = softmax_parts(logits, t)
    here, q, log_q, rel_q = teacher_parts(ids, teacher, vocab, t)
    safe = torch.where(here, ids, 0).long()
    gap = torch.where(q > 0, log_q - z.gather(1, safe) + lse[:, None], 0.0)
    some = here.any(-1)
    loss = w * t * t * (q * gap).sum(-1)
    loss_tol = w * t * t * ((q * (d[:, None] + rel_q + rel + 4 * U * gap.abs())).sum(-1) + (q * gap.abs() * (rel_q + 300 * U)).sum(-1))
    grad = torch.where(some[:, None], p, 0.0)
    tol = torch.where(some[:, None], p * rel, 0.0)
    grad.scatter_add_(1, safe, -q)
    tol.scatter_add_(1, safe, q * (rel_q + 64 * U))
    up = (w * dloss * t)[:, None]
    active = (w != 0)
    grad, tol = torch.where(active[:, None], grad * up, 0.0), torch.where(active[:, None], (tol + 4 * U * grad.abs()) * up.abs(), 0.0)
    fix = active & some
    return dict(loss=torch.where(fix, loss, 0.0), loss_tol=torch.where(fix, loss_tol + 4 * U * loss.abs(), 0.0), lse=torch.where(active, lse, 0.0),
                lse_tol=d, grad=grad, grad_tol=tol)


def expect(got, want, tol, dtype, what):
    close(got, want, tol + (want.abs() + tol) * HALF[dtype] + 1e-37, what)


def distill_data(rows, vocab, top, seed, dtype=F32, index=torch.int64, masked=True):
    gen = torch.Generator().manual_seed(seed)
    logits = (torch.randn(rows, vocab, generator=gen, dtype=F64) * 3).to(dtype)
    ids = torch.randint(0, vocab, (rows, top), generator=gen)
    if masked:
        ids = torch.where(torch.rand(rows, top, generator=gen) < 0.1, torch.randint(-2, 0, (rows, top), generator=gen), ids)
        ids = torch.where(torch.rand(rows, top, generator=gen) < 0.02, vocab, ids)
    teacher = (torch.randn(rows, top, generator=gen, dtype=F64) * 2).to(dtype)
    w = torch.where(torch.rand(rows, generator=gen) < 0.2, 0.0, torch.rand(rows, generator=gen) + 0.1)
    return logits, ids.to(index), teacher, w


def check_distill(fp, logits, ids, teacher, w, t=1.0, g_dtype=None, ld=None, offset=0, in_place=False, ld_t=None):
    rows, vocab = logits.shape
    g_dtype = g_dtype or logits.dtype
    dloss = torch.rand(rows, generator=torch.Generator().manual_seed(vocab)) + 0.5
    one = torch.ones(rows)
    wd = one if w is None else w
    ml = Matrix(rows, vocab, logits.dtype, ld, offset, logits)
    mt = Matrix(rows, ids.shape[1], teacher.dtype, ld_t, 0, teacher)
    mg = ml if in_place else Matrix(rows, vocab, g_dtype, ld, offset)
    dev = dict(weight=None if w is None else w.cuda(), temperature=t)
    loss, lse = (torch.full((rows,), 9.0, device="cuda") for _ in range(2))
    want = distill_reference(logits, ids, teacher, t, wd.double(), one.double())
    fp.fsdp_distill_loss_forward(ml.t, ids.cuda(), mt.t, loss, lse, **dev)
    expect(loss, want["loss"], want["loss_tol"], F32, "loss")
    expect(lse, want["lse"], want["lse_tol"], F32, "lse")
    loss2, lse2 = torch.empty_like(loss), torch.empty_like(lse)
    fp.fsdp_distill_loss_forward(ml.t, ids.cuda(), mt.t, loss2, lse2, dlogits=mg.t, **dev)
    expect(loss2, want["loss"], want["loss_tol"], F32, "loss with gradient")
    expect(lse2, want["lse"], want["lse_tol"], F32, "lse with gradient")
    expect(mg.t, want["grad"], want["grad_tol"], g_dtype, "dlogits of the forward call")
    if in_place:
        ml.t.copy_(logits)
    want = distill_reference(logits, ids, teacher, t, wd.double(), dloss.double())
    fp.fsdp_distill_loss_backward(ml.t, ids.cuda(), mt.t, lse, mg.t, dloss=dloss.cuda(), **dev)
    expect(mg.t, want["grad"], want["grad_tol"], g_dtype, "dlogits")
    fp.fsdp_ops_sync_status()
    assert mg.intact() and ml.intact() and mt.intact()


def policy_reference(logits, ids, old, ref, adv, t, w, dloss, low, high, kl):
    rows, vocab = logits.shape
    z, lse, p, d, rel = softmax_parts(logits, t)
    good = (ids >= 0) & (ids < vocab)
    safe = torch.where(good, ids, 0).long()[:, None]
    logp = z.gather(1, safe)[:, 0] - lse
    logp_tol = d + rel[:, 0] + 2 * U * logp.abs()
    gap_o = torch.zeros_like(logp) if old is None else logp - old.double()
    r = torch.exp(gap_o)
    r_rel = 0.0 if old is None else logp_tol + (4 + 4 * gap_o.abs()) * U
    held = r.clamp(1 - low, 1 + high)
    loss, tol = -torch.minimum(r * adv, held * adv), (r * r_rel + 4 * U * (r + held)) * adv.abs()
    c = torch.where(r * adv <= held * adv, -r * adv, torch.zeros_like(r))
    c_tol = tol
    if ref is not None:
        k = ref.double() - logp
        loss, tol = loss + kl * (torch.expm1(k) - k), tol + kl * (torch.expm1(k).abs() * logp_tol + 8 * U * (torch.exp(k) + k.abs() + 1))
        c, c_tol = c - kl * torch.expm1(k), c_tol + kl * (torch.exp(k) * (logp_tol + 4 * U) + 4 * U)
    grad = -p
    grad.scatter_add_(1, safe, torch.ones_like(safe, dtype=F64))
    g_tol = p * rel
    up = w * dloss / t
    fix = good & (w != 0)
    full = torch.where(fix[:, None], grad * (c * up)[:, None], 0.0)
    full_tol = torch.where(fix[:, None], (g_tol * c.abs()[:, None] + (grad.abs() + 2 * U) * (c_tol + 8 * U * c.abs())[:, None]) * up.abs()[:, None], 0.0)
    loss_tol = torch.where(fix, w * (tol + 4 * U * loss.abs()), 0.0)
    return dict(loss=torch.where(fix, w * loss, 0.0), loss_tol=loss_tol, logp=torch.where(fix, logp, 0.0), logp_tol=logp_tol,
                lse=torch.where(w != 0, lse, 0.0), lse_tol=d, grad=full, grad_tol=full_tol)


def policy_data(rows, vocab, seed, dtype=F32, index=torch.int64, t=1.0, low=0.2, high=0.3):
    gen = torch.Generator().manual_seed(seed)
    logits = (torch.randn(rows, vocab, generator=gen, dtype=F64) * 3).to(dtype)
    ids = torch.randint(0, vocab, (rows,), generator=gen)
    logp = torch.log_softmax(logits.double() / t, -1).gather(1, ids[:, None])[:, 0]
    drift = torch.randn(rows, generator=gen, dtype=F64) * 0.3
    for border in (math.log(max(1 - low, 1e-9)), math.log(1 + high)):  # the derivative jumps there
        drift = torch.where((drift - border).abs() < 1e-2, border + 2e-2, drift)
    old, ref = (logp - drift).float(), (logp - torch.randn(rows, generator=gen, dtype=F64) * 0.3).float()
    ids = torch.where(torch.rand(rows, generator=gen) < 0.1, torch.where(torch.rand(rows, generator=gen) < 0.5, -1, vocab), ids)
    adv = torch.randn(rows, generator=gen)
    w = torch.where(torch.rand(rows, generator=gen) < 0.2, 0.0, torch.rand(rows, generator=gen) + 0.1)
    return logits, ids.to(index), old, ref, adv, w


def check_policy(fp, logits, ids, old, ref, adv, w, t=1.0, low=0.2, high=0.3, kl=0.1, g_dtype=None, ld=None, offset=0, in_place=False):
    rows, vocab = logits.shape
    g_dtype = g_dtype or logits.dtype
    dloss = torch.rand(rows, generator=torch.Generator().manual_seed(vocab)) + 0.5
    one = torch.ones(rows)
    wd = (one if w is None else w).double()
    ml = Matrix(rows, vocab, logits.dtype, ld, offset, logits)
    mg = ml if in_place else Matrix(rows, vocab, g_dtype, ld, offset)
    cu = [None if v is None else v.cuda() for v in (old, ref, adv, w)]
    dev = dict(ref_logp=cu[1], weight=cu[3], temperature=t, clip_low=low, clip_high=high, kl=kl)
    want = policy_reference(logits, ids, old, ref, adv.double(), t, wd, one.double(), low, high, kl)
    out = [torch.full((rows,), 9.0, device="cuda") for _ in range(3)]
    fp.fsdp_policy_loss_forward(ml.t, ids.cuda(), cu[0], cu[2], *out, **dev)
    for got, n in zip(out, ("loss", "logp", "lse")):
        expect(got, want[n], want[n + "_tol"], F32, n)
    again = [torch.empty_like(v) for v in out]
    fp.fsdp_policy_loss_forward(ml.t, ids.cuda(), cu[0], cu[2], *again, dlogits=mg.t, **dev)
    for got, n in zip(again, ("loss", "logp", "lse")):
        expect(got, want[n], want[n + "_tol"], F32, n + " with gradient")
    expect(mg.t, want["grad"], want["grad_tol"], g_dtype, "dlogits of the forward call")
    if in_place:
        ml.t.copy_(logits)
    want = policy_reference(logits, ids, old, ref, adv.double(), t, wd, dloss.double(), low, high, kl)
    fp.fsdp_policy_loss_backward(ml.t, ids.cuda(), cu[0], cu[2], out[1], out[2], mg.t, dloss=dloss.cuda(), **dev)
    expect(mg.t, want["grad"], want["grad_tol"], g_dtype, "dlogits")
    fp.fsdp_ops_sync_status()
    assert mg.intact() and ml.intact()


VOCABS = [1, 2, 7, 8, 33, 100, 1000, 2047, 2048, 4096, 5001, 8200, 16384, 16392, 32768, 32771, 50021]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("vocab", VOCABS)
def test_distill(vocab, dtype):
    check_distill(fp_module(), *distill_data(9, vocab, 13, vocab, dtype))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("vocab", VOCABS)
def test_policy(vocab, dtype):
    check_policy(fp_module(), *policy_data(9, vocab, vocab, dtype))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("vocab", [65536, 100003, 131072, 262144, 262152, 600011])
def test_large_vocabularies(vocab, dtype):
    """Rows that several blocks share, and rows that no cluster holds."""
    check_distill(fp_module(), *distill_data(3, vocab, 40, 1, dtype), t=0.7)
    check_policy(fp_module(), *policy_data(3, vocab, 2, dtype))
    check_policy(fp_module(), *policy_data(3, vocab, 2, dtype), in_place=True)
    check_distill(fp_module(), *distill_data(3, vocab, 40, 1, dtype), in_place=True)


@pytest.mark.parametrize("rows", [0, 1, 2, 5, 153, 700, 3001])
@pytest.mark.parametrize("vocab", [96, 2051])
def test_rows(rows, vocab):
    check_distill(fp_module(), *distill_data(rows, vocab, 5, rows, BF16))
    check_policy(fp_module(), *policy_data(rows, vocab, rows, BF16))


@pytest.mark.parametrize("dtype,g_dtype", [(BF16, F32), (F32, BF16)])
@pytest.mark.parametrize("vocab", [512, 5001, 40000])
def test_gradient_types(vocab, dtype, g_dtype):
    check_distill(fp_module(), *distill_data(6, vocab, 9, 3, dtype), g_dtype=g_dtype)
    check_policy(fp_module(), *policy_data(6, vocab, 4, dtype), g_dtype=g_dtype)


@pytest.mark.parametrize("ld,offset", [(1000, 1), (1003, 0), (1008, 0), (1000, 8), (1001, 3)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_strides(ld, offset, dtype):
    check_distill(fp_module(), *distill_data(7, 1000, 9, ld, dtype), ld=ld, offset=offset, ld_t=11)
    check_policy(fp_module(), *policy_data(7, 1000, ld, dtype), ld=ld, offset=offset)
    check_policy(fp_module(), *policy_data(7, 1000, ld, dtype), ld=ld, offset=offset, in_place=True)


def test_gradient_of_another_phase():
    """Rows of logits and of the gradient that begin at different places within their 16-byte units."""
    fp = fp_module()
    logits, ids, teacher, w = distill_data(7, 999, 9, 5, BF16)
    ml, mg = Matrix(7, 999, BF16, 1003, 3, logits), Matrix(7, 999, BF16, 1001, 0)
    loss, lse = (torch.empty(7, device="cuda") for _ in range(2))
    fp.fsdp_distill_loss_forward(ml.t, ids.cuda(), teacher.cuda(), loss, lse, weight=w.cuda(), dlogits=mg.t)
    want = distill_reference(logits, ids, teacher, 1.0, w.double(), torch.ones(7, dtype=F64))
    expect(mg.t, want["grad"], want["grad_tol"], BF16, "dlogits")
    assert mg.intact() and ml.intact()


@pytest.mark.parametrize("top", [1, 2, 31, 33, 127, 128, 129, 500, 512, 513, 1024])
def test_tops(top):
    check_distill(fp_module(), *distill_data(5, 3000, top, top, BF16, torch.int32))


@pytest.mark.parametrize("vocab", [700, 40000])
def test_a_token_named_more_than_once(vocab):
    logits, ids, teacher, w = distill_data(6, vocab, 40, 8, F32)
    ids[0] = 3
    ids[1] = ids[1, :20].repeat(2)
    ids[2, 5], ids[2, 30] = vocab - 1, vocab - 1
    ids[3, ::3] = 0
    check_distill(fp_module(), logits, ids, teacher, None)


@pytest.mark.parametrize("t", [0.3, 2.0, 5.0])
def test_temperatures(t):
    check_distill(fp_module(), *distill_data(9, 1500, 20, 6, BF16), t=t)
    check_policy(fp_module(), *policy_data(9, 1500, 6, F32, t=t), t=t)


def test_rows_without_entries_and_without_weight():
    """No entry, entries of probability 0, a masked row full of NaN, all rows masked."""
    fp = fp_module()
    logits, ids, teacher, w = distill_data(8, 600, 6, 2, F32, masked=False)
    w = torch.ones(8)
    ids[0], teacher[1], ids[2, :5], teacher[3, 2:] = -1, -INF, -7, -INF
    w[4] = 0
    logits[4] = float("nan")
    logits[5, ids[5, 0]] = -INF  # a likely token that the student rules out: loss infinite, gradient finite
    teacher[6, 0], logits[6, ids[6, 0]] = -INF, -INF  # ruled out by both
    for vocab_pad in (0, 40001):
        z = torch.cat([logits, torch.full((8, vocab_pad), -INF)], 1)
        loss, lse, g = torch.empty(8, device="cuda"), torch.empty(8, device="cuda"), torch.empty_like(z, device="cuda")
        fp.fsdp_distill_loss_forward(z.cuda(), ids.cuda(), teacher.cuda(), loss, lse, weight=w.cuda(), dlogits=g)
        assert loss[:2].tolist() == [0.0, 0.0] and bool((g[[0, 1, 4]] == 0).all()) and loss[4] == 0 and lse[4] == 0
        assert loss[5] == INF and bool(torch.isfinite(g).all()) and bool(torch.isfinite(loss[[2, 3, 6, 7]]).all())
        want = distill_reference(torch.where(w[:, None] == 0, 0.0, z), ids, teacher, 1.0, w.double(), torch.ones(8, dtype=F64))
        expect(g, want["grad"], want["grad_tol"], F32, "dlogits")
        expect(loss, want["loss"], want["loss_tol"], F32, "loss")
        fp.fsdp_distill_loss_backward(z.cuda(), ids.cuda(), teacher.cuda(), lse, g, weight=w.cuda())
        expect(g, want["grad"], want["grad_tol"], F32, "dlogits of the backward call")
        fp.fsdp_distill_loss_forward(z.cuda(), ids.cuda(), teacher.cuda(), loss, lse, weight=torch.zeros(8, device="cuda"), dlogits=g)
        assert bool((g == 0).all()) and bool((loss == 0).all()) and bool((lse == 0).all())


@pytest.mark.parametrize("vocab", [600, 40001])
def test_specials(vocab):
    """A NaN or +infinity makes its row NaN and no other; a row of -infinity alone has no distribution; +-3e38 are values like others."""
    fp = fp_module()
    logits, ids, old, ref, adv, _ = policy_data(8, vocab, 12)
    ids = ids.clamp(0, vocab - 1)
    logits[0, 5], logits[1, vocab - 1], logits[2], logits[3, 7] = float("nan"), INF, -INF, 3e38
    logits[4], logits[4, 9] = -INF, float("nan")
    logits[5, 300:], ids[5] = -3e38, 5
    out = [torch.empty(8, device="cuda") for _ in range(3)]
    g = torch.empty(8, vocab, device="cuda")
    fp.fsdp_policy_loss_forward(logits.cuda(), ids.cuda(), old.cuda(), adv.cuda(), *out, ref_logp=ref.cuda(), kl=0.1, dlogits=g)
    assert bool(torch.isnan(g[[0, 1, 2, 4]]).all()) and bool(torch.isfinite(g[[5, 6, 7]]).all())
    assert bool(torch.isnan(out[2][[0, 1, 4]]).all()) and out[2][2] == -INF and out[2][3] == logits[3, 7]
    want = policy_reference(logits[6:], ids[6:], old[6:], ref[6:], adv[6:].double(), 1.0, torch.ones(2, dtype=F64), torch.ones(2, dtype=F64), 0.2, 0.2, 0.1)
    expect(g[6:], want["grad"], want["grad_tol"], F32, "dlogits")


def test_policy_without_old_or_reference():
    logits, ids, old, ref, adv, w = policy_data(20, 700, 3)
    check_policy(fp_module(), logits, ids, None, ref, adv, w)
    check_policy(fp_module(), logits, ids, old, None, adv, None)
    check_policy(fp_module(), logits, ids, None, None, adv, w, kl=0.0)
    check_policy(fp_module(), *policy_data(20, 700, 3, low=1e9, high=INF), low=INF, high=INF)
    check_policy(fp_module(), *policy_data(20, 700, 3, low=0.0, high=0.0), low=0.0, high=0.0)


def test_policy_at_the_border():
    """A ratio of exactly 1 with no room to clip: both terms are equal, and the gradient flows."""
    fp = fp_module()
    z = torch.zeros(2, 4, device="cuda")
    out = [torch.empty(2, device="cuda") for _ in range(3)]
    g = torch.empty_like(z)
    ids = torch.tensor([1, 2], device="cuda")
    fp.fsdp_policy_loss_forward(z, ids, None, torch.tensor([1.0, -1.0], device="cuda"), *out, clip_low=0.0, clip_high=0.0, dlogits=g)
    close(out[0], torch.tensor([-1.0, 1.0]), 1e-6, "loss")
    close(g, torch.tensor([[0.25, -0.75, 0.25, 0.25], [-0.25, -0.25, 0.75, -0.25]]), 1e-6, "dlogits")


def test_gradients_against_differences():
    """Central differences along random directions in 32 bits; a step of 2^-6 leaves third-order terms below 1e-3 of the inner
    product's scale, outputs' roundings less."""
    fp = fp_module()
    logits, ids, teacher, w = distill_data(12, 300, 7, 4)
    z, v = logits.cuda(), normals(1, 12, 300).float().cuda()
    _, tok, old, ref, adv, _ = policy_data(12, 300, 4)
    tok = tok.clamp(0, 299)

    def distill(e, g=None):
        loss, lse = torch.empty(12, device="cuda"), torch.empty(12, device="cuda")
        fp.fsdp_distill_loss_forward(z + e * v, ids.cuda(), teacher.cuda(), loss, lse, temperature=1.5, weight=w.cuda(), dlogits=g)
        return float(loss.double().sum())

    def policy(e, g=None):
        out = [torch.empty(12, device="cuda") for _ in range(3)]
        fp.fsdp_policy_loss_forward(z + e * v, tok.cuda(), old.cuda(), adv.cuda(), *out, ref_logp=ref.cuda(), kl=0.1, clip_low=INF, clip_high=INF, dlogits=g)
        return float(out[0].double().sum())

    for f in (distill, policy):
        g = torch.empty_like(z)
        f(0.0, g)
        want, scale = float((g.double() * v.double()).sum()), float((g.double() * v.double()).abs().sum())
        got = (f(2.0 ** -6) - f(-2.0 ** -6)) * 2.0 ** 5
        assert abs(got - want) <= 3e-3 * scale


@pytest.mark.parametrize("vocab", [1000, 100000])
def test_same_bits_streams_graphs_and_threads(vocab):
    fp = fp_module()
    logits, ids, teacher, w = (t.cuda() for t in distill_data(300, vocab, 20, 1, BF16))

    def outputs():
        return [torch.empty(300, device="cuda") for _ in range(2)] + [torch.empty_like(logits) for _ in range(2)]

    def go(o, stream=None):
        fp.fsdp_distill_loss_forward(logits, ids, teacher, o[0], o[1], weight=w, dlogits=o[2], stream=stream)
        fp.fsdp_distill_loss_backward(logits, ids, teacher, o[1], o[3], weight=w, stream=stream)

    first, again = outputs(), outputs()
    go(first)
    go(again)
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go(again)
    for t in again:
        t.fill_(7)
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    got = [outputs(), outputs()]
    torch.cuda.synchronize()

    def many(k):
        s = torch.cuda.Stream()
        for _ in range(10):
            go(got[k], s)
        s.synchronize()

    threads = [threading.Thread(target=many, args=(k,)) for k in range(2)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    for k in range(2):
        assert all(torch.equal(a, b) for a, b in zip(first, got[k]))
    fp.fsdp_ops_sync_status()


def test_binding_refusals():
    fp = fp_module()
    z, v = torch.empty(4, 50, device="cuda"), torch.empty(4, device="cuda")
    ids, t = torch.zeros(4, 3, dtype=torch.int64, device="cuda"), torch.empty(4, 3, device="cuda")
    bad = [((z, ids, t, v, None), {}, "lse is needed"), ((z, ids[:3], t, v, v), {}, "not 4"), ((z, ids, t[:, :2], v, v), {}, "not 4 x 3"),
           ((z, ids.float(), t, v, v), {}, "not one of"), ((z, ids, t, v[:3], v), {}, "vector"), ((z.half(), ids, t, v, v), {}, "float16"),
           ((z, ids, t, v, v), dict(dlogits=z[:, :49]), "not 4 x 50"), ((z, ids, t, v, v), dict(weight=v.to(BF16)), "bfloat16")]
    for args, kw, word in bad:
        with pytest.raises(ValueError, match=word):
            fp.fsdp_distill_loss_forward(*args, **kw)
    for bad_t in (0.0, -1.0, INF, float("nan"), 1e-45):
        with pytest.raises(fp.FsdpError, match="temperature"):
            fp.fsdp_distill_loss_forward(z, ids, t, v, v, temperature=bad_t)
    with pytest.raises(fp.FsdpError, match="FSDP_DISTILL_MAX_TOP"):
        fp.fsdp_distill_loss_forward(z, torch.zeros(4, 1025, dtype=torch.int64, device="cuda"), torch.empty(4, 1025, device="cuda"), v, v)
    tok = ids[:, 0].contiguous()
    with pytest.raises(ValueError, match="advantage is needed"):
        fp.fsdp_policy_loss_forward(z, tok, v, None, v, v, v)
    with pytest.raises(ValueError, match="tokens for"):
        fp.fsdp_policy_loss_forward(z, tok[:2], v, v, v, v, v)
    for kw, word in ((dict(clip_low=-0.1), "clip_low"), (dict(clip_high=float("nan")), "clip_high"), (dict(kl=-1.0), "kl"), (dict(kl=INF), "kl")):
        with pytest.raises(fp.FsdpError, match=word):
            fp.fsdp_policy_loss_forward(z, tok, v, v, v, v, v, **kw)
    with pytest.raises(fp.FsdpError, match="dlogits is logits"):
        fp.fsdp_policy_loss_forward(z, tok, v, v, v, v, v, dlogits=z.view(BF16)[:, :50])


MANY = 1000  # rows, of which short ones go to a warp each


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("vocab", [1, 7, 33, 512, 513, 1021, 2048, 2049, 4089, 4096])
def test_many_short_rows(vocab, dtype):
    check_distill(fp_module(), *distill_data(MANY, vocab, 13, vocab, dtype), t=0.8)
    check_policy(fp_module(), *policy_data(MANY, vocab, vocab, dtype, t=0.8), t=0.8)


@pytest.mark.parametrize("ld,offset", [(1000, 1), (1003, 0), (1008, 8), (1001, 3)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_many_short_rows_apart(ld, offset, dtype):
    other = F32 if dtype == BF16 else BF16
    check_distill(fp_module(), *distill_data(MANY, 1000, 9, ld, dtype), ld=ld, offset=offset, ld_t=11, g_dtype=other)
    check_distill(fp_module(), *distill_data(MANY, 1000, 9, ld, dtype), ld=ld, offset=offset, in_place=True)
    check_policy(fp_module(), *policy_data(MANY, 1000, ld, dtype), ld=ld, offset=offset, g_dtype=other)
    check_policy(fp_module(), *policy_data(MANY, 1000, ld, dtype), ld=ld, offset=offset, in_place=True)


@pytest.mark.parametrize("top", [1, 32, 33, 128, 129])
def test_tops_of_many_short_rows(top):
    check_distill(fp_module(), *distill_data(MANY, 300, top, top, BF16, torch.int32))


def test_tokens_named_more_than_once_in_many_short_rows():
    logits, ids, teacher, w = distill_data(MANY, 700, 40, 8, F32)
    ids[::4] = 3
    ids[1::4] = ids[1::4, :20].repeat(1, 2)
    ids[2::4, 5], ids[2::4, 30] = 699, 699
    ids[3::4, ::3] = 0
    check_distill(fp_module(), logits, ids, teacher, None)


def test_specials_in_many_short_rows():
    """The rows of ``test_specials`` and of ``test_rows_without_entries_and_without_weight``, over and over."""
    fp = fp_module()
    n = MANY // 8
    logits, ids, old, ref, adv, _ = policy_data(8, 600, 12)
    ids = ids.clamp(0, 599)
    logits[0, 5], logits[1, 599], logits[2], logits[3, 7] = float("nan"), INF, -INF, 3e38
    logits[4], logits[4, 9] = -INF, float("nan")
    logits[5, 300:], ids[5] = -3e38, 5
    g = torch.empty(8 * n, 600, device="cuda")
    out = [torch.empty(8 * n, device="cuda") for _ in range(3)]
    many = [v.repeat(n, *[1] * (v.dim() - 1)).cuda() for v in (logits, ids, old, ref, adv)]
    fp.fsdp_policy_loss_forward(many[0], many[1], many[2], many[4], *out, ref_logp=many[3], kl=0.1, dlogits=g)
    first = torch.arange(0, 8 * n, 8)
    assert all(bool(torch.isnan(g[first + r]).all()) for r in (0, 1, 2, 4)) and all(bool(torch.isfinite(g[first + r]).all()) for r in (5, 6, 7))
    assert all(bool(torch.isnan(out[2][first + r]).all()) for r in (0, 1, 4))
    assert bool((out[2][first + 2] == -INF).all()) and bool((out[2][first + 3] == logits[3, 7].item()).all())

    logits, ids, teacher, w = distill_data(8, 600, 6, 2, F32, masked=False)
    w = torch.ones(8)
    ids[0], teacher[1], ids[2, :5], teacher[3, 2:] = -1, -INF, -7, -INF
    w[4], logits[4], logits[5, ids[5, 0]] = 0, float("nan"), -INF
    teacher[6, 0], logits[6, ids[6, 0]] = -INF, -INF
    want = distill_reference(torch.where(w[:, None] == 0, 0.0, logits), ids, teacher, 1.0, w.double(), torch.ones(8, dtype=F64))
    want = {k: v.repeat(n, *[1] * (v.dim() - 1)) for k, v in want.items()}
    many = [v.repeat(n, *[1] * (v.dim() - 1)).cuda() for v in (logits, ids, teacher, w)]
    loss, lse = (torch.empty(8 * n, device="cuda") for _ in range(2))
    fp.fsdp_distill_loss_forward(*many[:3], loss, lse, weight=many[3], dlogits=g)
    expect(g, want["grad"], want["grad_tol"], F32, "dlogits")
    expect(loss, want["loss"], want["loss_tol"], F32, "loss")
    assert bool((lse[first + 4] == 0).all())
    fp.fsdp_distill_loss_backward(*many[:3], lse, g, weight=many[3])
    expect(g, want["grad"], want["grad_tol"], F32, "dlogits of the backward call")


@pytest.mark.parametrize("vocab,top", [(13000, 64), (13100, 64), (13184, 9), (26200, 64), (40000, 216), (40000, 230), (131072, 240)])
def test_rings_that_nearly_fill_an_sm(vocab, top):
    """Slices and teacher's entries of which three or four take 106 to 108 KB: one stage fewer."""
    check_distill(fp_module(), *distill_data(5, vocab, top, 1, BF16, torch.int32))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("vocab", [4097, 8191, 8192, 8193, 16384])
def test_many_rows_of_several_warps(vocab, dtype):
    vocab = vocab if dtype == BF16 else vocab // 2
    check_distill(fp_module(), *distill_data(700, vocab, 40, vocab, dtype), t=0.8)
    check_policy(fp_module(), *policy_data(700, vocab, vocab, dtype, t=0.8), t=0.8)


@pytest.mark.parametrize("vocab", [5001, 15001])
def test_many_rows_of_several_warps_apart(vocab):
    """Rows that begin anywhere, in place and in another type, entries that name a token again."""
    logits, ids, teacher, w = distill_data(700, vocab, 100, vocab, BF16)
    ids[::3, 50:] = ids[::3, :50]
    ids[1::3] = vocab - 1
    check_distill(fp_module(), logits, ids, teacher, w, ld=vocab + 4, offset=3, ld_t=101, in_place=True)
    check_distill(fp_module(), logits, ids, teacher, None, ld=vocab + 2, offset=1, g_dtype=F32)
    check_policy(fp_module(), *policy_data(700, vocab, 5, BF16), ld=vocab + 4, offset=3, in_place=True)


@pytest.mark.parametrize("rows", [20, 38, 61, 76, 152, 305])
def test_rows_for_clusters_of_every_size(rows):
    check_distill(fp_module(), *distill_data(rows, 33001, 20, rows, BF16))
    check_policy(fp_module(), *policy_data(rows, 33001, rows, BF16))

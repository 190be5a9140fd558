"""Losses of rows whose vocabulary is masked with large finite logits, of the type's lowest value or short of it: those are values
like others.  Against the definitions in 64 bits.

Tolerances, in units u = 2^-24.  Exponents are differences to the row's maximum: exact or rounded once, scaled once, off by at most 4 u of
their size, which for an exponential that is not 0 is below 104; so with Z = min(largest (maximum - z) / T, 104) + 1 an exponential is
off by 8 Z u relative, sums of them by 256 u more (chains of at most 256 additions), and the logarithm of a sum and each
probability by d = (8 Z + 270) u.  lse adds maximum / T and is rounded to 2 u of its own size.  A log-probability is a
scaled difference less that logarithm.  A gradient from lse alone takes its rounding too, 3 |lse| u relative."""
import pytest
import torch

from gpu_util import fp_module
from ops_util import BF16, EPS32, F32, F64, HALF, Matrix, close

pytestmark = pytest.mark.gpu
U = EPS32
INF = float("inf")
LOW = {F32: torch.finfo(F32).min, BF16: torch.finfo(BF16).min}
SHAPES = [(600, 3), (600, 1300), (5001, 3), (5001, 700), (12000, 650), (40001, 3), (131072, 4)]


def parts(logits, t):
    """Scaled differences to a row's maximum, the logarithm of their exponentials' sum, p, the tolerance of both, lse and its own."""
    top = logits.double().amax(-1, keepdim=True)
    z = (logits.double() - top) / t
    log_sum = torch.logsumexp(z, -1, keepdim=True)
    near = torch.where(z > -104, -z, 0.0).amax(-1, keepdim=True) + 1
    lse = (top / t + log_sum)[:, 0]
    d = (8 * near + 270) * U
    return z, log_sum, torch.exp(z - log_sum), d, lse, d[:, 0] + 3 * U * lse.abs()


def expect(got, want, tol, what):
    close(got, want, tol + (want.abs() + tol) * HALF[got.dtype] + 1e-37, what)


def masked(rows, vocab, mask, dtype, seed):
    """A run of a fifth of the vocabulary stays; of row 1 one token, of row 0 none; and where each row's begins."""
    gen = torch.Generator().manual_seed(seed)
    logits = (torch.randn(rows, vocab, generator=gen, dtype=F64) * 3).to(dtype)
    first = torch.randint(0, vocab - vocab // 5, (rows, 1), generator=gen)
    n = torch.full((rows, 1), vocab // 5)
    n[0], n[1] = 0, 1
    j = torch.arange(vocab)
    return torch.where((j >= first) & (j < first + n), logits, torch.tensor(mask, dtype=dtype)), first, n, gen


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("mask", [-1e4, -1e9, -1e10, -1e20, -1e30, "lowest"])
def test_policy(mask, dtype, shape):
    fp = fp_module()
    vocab, rows = shape
    value = LOW[dtype] if mask == "lowest" else mask
    logits, first, n, gen = masked(rows, vocab, value, dtype, vocab)
    ids = first[:, 0] + (torch.rand(rows, generator=gen) * n[:, 0]).long()  # of row 0 any token
    adv, dloss = torch.randn(rows, generator=gen), torch.rand(rows, generator=gen) + 0.5
    for t in (0.7, 1.0):
        z, log_sum, p, d, lse, lse_tol = parts(logits, t)
        logp = (z.gather(1, ids[:, None]) - log_sum)[:, 0]
        logp_tol = d[:, 0] + 4 * U * logp.abs()
        want = p.clone()
        want.scatter_add_(1, ids[:, None], torch.full((rows, 1), -1.0, dtype=F64))
        tol = p * (2 * d + 16 * U) + 4 * U * want.abs()
        ml, mg = Matrix(rows, vocab, dtype, None, 0, logits), Matrix(rows, vocab, dtype)
        loss, got_p, got_l = (torch.empty(rows, device="cuda") for _ in range(3))
        for g in (None, mg.t):
            fp.fsdp_policy_loss_forward(ml.t, ids.cuda(), None, adv.cuda(), loss, got_p, got_l, temperature=t, dlogits=g)
            expect(loss, -adv.double(), 4 * U * adv.abs().double(), "loss")
            expect(got_p, logp, logp_tol, "logp")
            if abs(value) / t < 3e38:
                expect(got_l, lse, lse_tol, "lse")
        by = (adv.double() / t)[:, None]
        expect(mg.t, want * by, (tol + 4 * U * want.abs()) * by.abs(), "dlogits of the forward call")
        # From lse: not row 0, whose lse cannot say how many tokens share its maximum.
        fp.fsdp_policy_loss_backward(ml.t, ids.cuda(), None, adv.cuda(), got_p, got_l, mg.t, temperature=t, dloss=dloss.cuda())
        by = by * dloss.double()[:, None]
        tol = tol + p * 6 * U * lse.abs()[:, None]
        expect(mg.t[1:], (want * by)[1:], ((tol + 8 * U * want.abs()) * by.abs())[1:], "dlogits")
        assert ml.intact() and mg.intact()
    fp.fsdp_ops_sync_status()


def check_distill(rows, vocab, logits, ids, teacher, t, lse_counts, named_tol=0.0):
    """Loss, lse and gradients against the definition; the gradient from lse of rows where that counts."""
    fp = fp_module()
    z, log_sum, p, d, lse, lse_tol = parts(logits, t)
    here = (ids >= 0) & (teacher.double() > -INF)
    v = torch.where(here, teacher.double(), -INF)
    v = (v - v.amax(-1, keepdim=True)) / t
    log_q = torch.where(here, v - torch.logsumexp(v, -1, keepdim=True), 0.0)
    q = torch.where(here, torch.exp(log_q), 0.0)
    rel_q = (8 * (torch.where(v > -104, -v, 0.0).amax(-1, keepdim=True) + 1) + 270) * U
    safe = torch.where(here, ids, 0).long()
    gap = torch.where(q > 0, log_q - z.gather(1, safe) + log_sum, 0.0)
    loss = t * t * (q * gap).sum(-1)
    # Terms log q, (z - maximum) / T and log sum, each rounded to a few u of its size and weighed by a q that is off by rel_q.
    size = torch.where(q > 0, log_q.abs() + z.gather(1, safe).abs() + log_sum.abs(), 0.0)
    loss_tol = t * t * ((q * size).sum(-1) * (2 * rel_q[:, 0] + 16 * U) + 2 * d[:, 0] + 2 * rel_q[:, 0])
    want = p.clone()
    want.scatter_add_(1, safe, -q)
    tol = p * (2 * d + 16 * U)
    tol.scatter_add_(1, safe, q * (2 * rel_q + 64 * U))
    want, tol = want * t, (tol + 4 * U * want.abs()) * t
    some = here.any(-1)
    want, tol = torch.where(some[:, None], want, 0.0), torch.where(some[:, None], tol, 0.0)
    loss = torch.where(some, loss, 0.0)
    ml, mg = Matrix(rows, vocab, logits.dtype, None, 0, logits), Matrix(rows, vocab, logits.dtype)
    mt = teacher.cuda()
    got, got_l = (torch.empty(rows, device="cuda") for _ in range(2))
    for g in (None, mg.t):
        fp.fsdp_distill_loss_forward(ml.t, ids.cuda(), mt, got, got_l, temperature=t, dlogits=g)
        expect(got, loss, loss_tol, "loss")
        if float(logits.double().abs().max()) / t < 3e38:
            expect(got_l, lse, lse_tol, "lse")
    expect(mg.t, want, tol, "dlogits of the forward call")
    fp.fsdp_distill_loss_backward(ml.t, ids.cuda(), mt, got_l, mg.t, temperature=t)
    tol = tol + p * (6 * U * t) * lse.abs()[:, None]
    expect(mg.t[lse_counts], want[lse_counts], tol[lse_counts], "dlogits")
    fp.fsdp_ops_sync_status()
    assert ml.intact() and mg.intact()


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("mask", [-1e4, -1e9, -1e10, -1e20, -1e30, "lowest"])
def test_distill(mask, dtype, shape):
    vocab, rows = shape
    value = LOW[dtype] if mask == "lowest" else mask
    logits, first, n, gen = masked(rows, vocab, value, dtype, vocab + 1)
    top = 9
    ids = first + (torch.rand(rows, top, generator=gen) * n).long()  # within the run; of rows 0 and 1 one token, named again and again
    ids[0] = torch.arange(top) * (vocab // top)
    teacher = (torch.randn(rows, top, generator=gen, dtype=F64) * 2).to(dtype)
    if mask != "lowest":  # a token that the student rules out: a large loss
        ids[2, 4] = (first[2, 0] + vocab // 2) % vocab
    for t in (0.7, 1.0):
        check_distill(rows, vocab, logits, ids, teacher, t, slice(1, None))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("vocab", [600, 40001])
@pytest.mark.parametrize("offset", [-3e4, 1e3, 2e5])
def test_far_offsets(offset, vocab, dtype):
    """All of a row's logits around a number that is large beside their differences."""
    gen = torch.Generator().manual_seed(vocab)
    logits = (torch.randn(5, vocab, generator=gen, dtype=F64) * abs(offset) / 1e3 + offset).to(dtype)
    ids = torch.randint(0, vocab, (5, 20), generator=gen)
    check_distill(5, vocab, logits, ids, torch.randn(5, 20, generator=gen, dtype=F64).to(dtype), 1.0, slice(0, 5))


@pytest.mark.parametrize("vocab", [600, 40001])
def test_rows_of_infinities(vocab):
    """A row of -infinity alone has no distribution: its loss and gradient are NaN, and no other row's."""
    fp = fp_module()
    logits = torch.randn(4, vocab, generator=torch.Generator().manual_seed(1))
    logits[1], logits[2, 3] = -INF, INF
    ids = torch.arange(12).reshape(4, 3)
    loss, lse = (torch.empty(4, device="cuda") for _ in range(2))
    g = torch.empty(4, vocab, device="cuda")
    for d in (None, g):
        fp.fsdp_distill_loss_forward(logits.cuda(), ids.cuda(), torch.zeros(4, 3, device="cuda"), loss, lse, dlogits=d)
        assert torch.isnan(loss).tolist() == [False, True, True, False] and lse[1] == -INF
    assert bool(torch.isnan(g[1:3]).all()) and bool(torch.isfinite(g[[0, 3]]).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("top", [5, 128, 129, 700])
@pytest.mark.parametrize("t", [0.5, 0.7, 1.0])
def test_masked_teachers(t, top, dtype):
    """A teacher's logits of the type's lowest value, throughout or in part, and of its highest: values like others, which count."""
    gen = torch.Generator().manual_seed(top)
    logits = torch.randn(6, 3000, generator=gen, dtype=F64).to(dtype)
    ids = torch.stack([torch.randperm(3000, generator=gen)[:top] for _ in range(6)])
    teacher = torch.randn(6, top, generator=gen, dtype=F64).to(dtype)
    teacher[0], teacher[1, 1:], teacher[2, ::2], teacher[3, top - 1] = LOW[dtype], LOW[dtype], LOW[dtype], -LOW[dtype]
    teacher[4, :] = -1e30
    check_distill(6, 3000, logits, ids, teacher, t, slice(0, 6))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("vocab,rows", [(600, 5), (600, 1300), (16000, 5), (40001, 5), (131072, 4), (600, 0)])
def test_no_entries(vocab, rows, dtype):
    """A batch whose rows have no teacher's entries at all: losses and gradients of 0, and their lse."""
    fp = fp_module()
    logits = torch.randn(rows, vocab, generator=torch.Generator().manual_seed(2), dtype=F64).to(dtype)
    ids, teacher = torch.empty(rows, 0, dtype=torch.int64, device="cuda"), torch.empty(rows, 0, device="cuda")
    loss, lse = (torch.full((rows,), 9.0, device="cuda") for _ in range(2))
    for g in (None, torch.full((rows, vocab), 9.0, dtype=dtype, device="cuda")):
        fp.fsdp_distill_loss_forward(logits.cuda(), ids, teacher, loss, lse, dlogits=g)
        assert bool((loss == 0).all())
        if rows:
            *_, want, tol = parts(logits, 1.0)
            expect(lse, want, tol, "lse")
    assert bool((g == 0).all())
    g.fill_(9.0)
    fp.fsdp_distill_loss_backward(logits.cuda(), ids, teacher, lse, g)
    assert bool((g == 0).all())
    fp.fsdp_ops_sync_status()


def test_no_entries_refusals():
    fp = fp_module()
    z, loss, lse = torch.randn(5, 100, device="cuda"), torch.empty(5, device="cuda"), torch.empty(5, device="cuda")
    ids, teacher = torch.empty(5, 0, dtype=torch.int64, device="cuda"), torch.empty(5, 0, device="cuda")
    for bad, t, word in ((ids[:4], teacher, "4 x 0"), (ids.float(), teacher, "float32"), (ids, teacher[:3], "3 x 0"), (ids, teacher.double(), "float64"),
                         (ids, torch.empty(5, 2, device="cuda"), "5 x 2"), (torch.zeros(5, 2, dtype=torch.int64, device="cuda"), teacher, "5 x 0"),
                         (ids.cpu(), teacher, "not a CUDA tensor"), (ids, teacher.cpu(), "not a CUDA tensor"), (ids[0], teacher, "dimensions"),
                         (None, teacher, "not a tensor")):
        with pytest.raises(ValueError, match=word):
            fp.fsdp_distill_loss_forward(z, bad, t, loss, lse)


@pytest.mark.parametrize("vocab,rows", [(600, 3), (5001, 700), (12000, 650), (40001, 3), (131072, 4)])
def test_both_ends_of_the_range(vocab, rows):
    """A student's maximum and a named token's logit further apart than binary32 reaches, at a small q: the loss lies within it."""
    fp = fp_module()
    logits = torch.randn(rows, vocab, generator=torch.Generator().manual_seed(3))
    logits[:, 7], logits[:, vocab - 5] = 3e38, -3e38
    ids = torch.tensor([[7, vocab - 5, 11]]).expand(rows, 3).contiguous()
    teacher = torch.tensor([[8.0, 0.0, float("-inf")]]).expand(rows, 3).contiguous()
    q = torch.softmax(teacher[0].double(), -1)
    want = (q[1] * (logits[:, vocab - 5].double() - logits[:, 7].double()).abs())
    loss, lse = (torch.empty(rows, device="cuda") for _ in range(2))
    g = torch.empty(rows, vocab, device="cuda")
    for d in (None, g):
        fp.fsdp_distill_loss_forward(logits.cuda(), ids.cuda(), teacher.cuda(), loss, lse, dlogits=d)
        expect(loss, want, want * 400 * U, "loss")  # an exponential of 8 (64 + 4 u), a quotient, a product and roundings of sums
    for j, value in ((7, 1 - q[0]), (vocab - 5, -q[1]), (11, 0.0)):
        expect(g[:, j], torch.full((rows,), float(value), dtype=F64), 400 * U, f"dlogits of token {j}")

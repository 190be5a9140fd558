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

"""The embedding, the recurrence and the losses on matrices of more than 2^31 elements, whose last rows are compared with the same
rows computed alone; waits that give up; and everything in one captured graph."""
import pytest
import torch

from gpu_util import fp_module
from ops_util import BF16, F32

pytestmark = pytest.mark.gpu


def rows_of(rows, cols, seed, dtype=BF16, std=1.0):
    """Rows that repeat every 1,031 and differ by a factor of 2 at the end, without a large temporary."""
    base = (torch.randn(1031, cols, generator=torch.Generator().manual_seed(seed)) * std).to(dtype).cuda()
    out = torch.empty(rows, cols, dtype=dtype, device="cuda")
    for at in range(0, rows, 1031):
        n = min(1031, rows - at)
        out[at:at + n] = base[:n]
    out[-5:] *= 2
    return out


@pytest.mark.parametrize("cols", [32768, 32767])
def test_embedding_beyond_32_bits(cols):
    """A table of 66,001 rows and a batch of 70,003: rows of both lie behind 2^31 elements."""
    fp = fp_module()
    vocab, rows = 66001, 70003
    table = rows_of(vocab, cols, 1)
    tokens = torch.arange(rows, device="cuda") * 31 % vocab
    tokens[-7:] = torch.tensor([vocab - 1, 0, vocab - 2, -1, vocab, 17, vocab - 1], device="cuda")
    out = torch.empty(rows, cols, dtype=BF16, device="cuda")
    fp.fsdp_embedding_forward(tokens, table, out, scale=0.5)
    want = torch.where(((tokens >= 0) & (tokens < vocab))[-7:, None], table[tokens[-7:].clamp(0, vocab - 1)] * 0.5, 0.0)
    assert torch.equal(out[-7:], want) and torch.equal(out[:7], table[tokens[:7]] * 0.5)
    # The gradient of the same rows: sums of a token's rows, here of values that sum exactly.
    out.copy_(out.float().mul_(8).round_().clamp_(-64, 64))
    grad = torch.empty_like(table)
    fp.fsdp_embedding_backward(tokens, out, grad)
    for v in (0, 5, vocab - 2, vocab - 1):
        rows_v = (tokens == v).nonzero()[:, 0]
        assert torch.equal(grad[v], out[rows_v].float().sum(0).to(BF16))
    grad2 = grad.clone()
    fp.fsdp_embedding_backward(tokens[:0], out[:0], grad2, accumulate=True)
    assert torch.equal(grad2[-3:], grad[-3:])


@pytest.mark.parametrize("cols", [32768, 32767])
def test_scan_beyond_32_bits(cols):
    fp = fp_module()
    rows, tail = 66001, 66001 % 128
    x, gate, dh = rows_of(rows, cols, 2), rows_of(rows, cols, 3), rows_of(rows, cols, 4, std=0.1)
    bias = torch.rand(cols, device="cuda") * 3
    off = torch.tensor([0, 100, rows - tail, rows], device="cuda")

    def both(x, gate, dh, off):
        n = x.shape[0]
        h, dx, dg, db = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x), torch.empty_like(bias)
        states = torch.empty(fp.fsdp_gated_scan_states(n, cols), cols, device="cuda")
        fp.fsdp_gated_scan_forward(x, gate, h, bias=bias, offsets=off, states=states)
        fp.fsdp_gated_scan_backward(dh, x, gate, states, dx, dg, bias=bias, dbias=db, offsets=off)
        return h, dx, dg

    whole = both(x, gate, dh, off)
    last = both(x[-tail:].clone(), gate[-tail:].clone(), dh[-tail:].clone(), torch.tensor([0, tail], device="cuda"))
    fp.fsdp_ops_sync_status()
    for p, q in zip(whole, last):
        assert torch.equal(p[-tail:], q)


@pytest.mark.parametrize("vocab", [131072, 131071])
def test_losses_beyond_32_bits(vocab):
    fp = fp_module()
    rows = 17001
    z = rows_of(rows, vocab, 5, std=2.0)
    ids = torch.arange(rows, device="cuda")[:, None] * 77 % (vocab - 40) + torch.arange(33, device="cuda")
    teacher = torch.randn(rows, 33, device="cuda")
    adv = torch.randn(rows, device="cuda")

    def distill(z, ids, teacher):
        n = z.shape[0]
        loss, lse, g = torch.empty(n, device="cuda"), torch.empty(n, device="cuda"), torch.empty_like(z)
        fp.fsdp_distill_loss_forward(z, ids, teacher, loss, lse, dlogits=g)
        g2 = torch.empty_like(z)
        fp.fsdp_distill_loss_backward(z, ids, teacher, lse, g2)
        return loss, lse, g[-7:].clone(), g2[-7:].clone()

    def policy(z, tok, adv):
        n = z.shape[0]
        out, g = [torch.empty(n, device="cuda") for _ in range(3)], torch.empty_like(z)
        fp.fsdp_policy_loss_forward(z, tok, None, adv, *out, dlogits=g)
        return (*out, g[-7:].clone())

    for f, args in ((distill, (ids, teacher)), (policy, (ids[:, 3].contiguous(), adv))):
        whole, last = f(z, *args), f(z[-7:], *(a[-7:] for a in args))
        fp.fsdp_ops_sync_status()
        for p, q in zip(whole, last):
            # Another cut of a row into slices may round its sum the other way.
            assert bool(((p[-7:].float() - q.float()).abs() <= q.float().abs() * 2 ** -7 + 1e-6).all())


def test_scan_wait_that_gives_up():
    """The first tile keeps its state to itself: the tiles behind it give up, say so, and the next call is whole again."""
    fp = fp_module()
    x, gate = torch.randn(3000, 200, device="cuda"), torch.randn(3000, 200, device="cuda") + 4
    states = torch.empty(fp.fsdp_gated_scan_states(3000, 200), 200, device="cuda")

    def forward():
        h = torch.empty_like(x)
        fp.fsdp_gated_scan_forward(x, gate, h, seq_len=3000, states=states)
        return h

    def backward():
        dx, dg = torch.empty_like(x), torch.empty_like(x)
        fp.fsdp_gated_scan_backward(x, x, gate, states, dx, dg, seq_len=3000)
        return dx

    h, dx = forward(), backward()
    fp.fsdp_ops_sync_status()
    fp.fsdp_debug_set_wait_fault(1, 20_000_000)
    try:
        for call in (backward, forward):
            call()
            with pytest.raises(fp.FsdpError, match="gave up"):
                fp.fsdp_ops_sync_status()
    finally:
        fp.fsdp_debug_set_wait_fault(0, 0)
    again = forward(), backward()
    fp.fsdp_ops_sync_status()
    assert torch.equal(again[0], h) and torch.equal(again[1], dx)


@pytest.mark.parametrize("rows,vocab", [(40, 3000), (300, 3000), (5, 40000), (300, 40000)])
def test_loss_wait_that_gives_up(rows, vocab):
    """A block's first slice never comes, with and without a cluster that shares its row."""
    fp = fp_module()
    z = torch.randn(rows, vocab, device="cuda")
    ids, t = torch.arange(9, device="cuda").repeat(rows, 1), torch.randn(rows, 9, device="cuda")
    adv = torch.randn(rows, device="cuda")

    def distill():
        loss, lse, g = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda"), torch.empty_like(z)
        fp.fsdp_distill_loss_forward(z, ids, t, loss, lse, dlogits=g if vocab == 3000 else None)  # of short rows a loss alone waits for nothing
        return loss, lse

    def policy():
        out, g = [torch.empty(rows, device="cuda") for _ in range(3)], torch.empty_like(z)
        fp.fsdp_policy_loss_forward(z, ids[:, 1].contiguous(), None, adv, *out, dlogits=g)
        return (*out, g)

    lse = distill()[1]

    def gradient():
        g = torch.empty_like(z)
        fp.fsdp_distill_loss_backward(z, ids, t, lse, g)
        return (g,)

    first = [f() for f in (distill, policy, gradient)]
    fp.fsdp_ops_sync_status()
    fp.fsdp_debug_set_wait_fault(1, 20_000_000)
    try:
        for f in (distill, policy, gradient):
            f()
            with pytest.raises(fp.FsdpError, match="gave up"):
                fp.fsdp_ops_sync_status()
    finally:
        fp.fsdp_debug_set_wait_fault(0, 0)
    again = [f() for f in (distill, policy, gradient)]
    fp.fsdp_ops_sync_status()
    for p, q in zip(first, again):
        assert all(torch.equal(a, b) for a, b in zip(p, q))


def test_a_step_in_one_graph():
    """Lookup, recurrence, loss and all their gradients captured into one graph, replayed on other inputs."""
    fp = fp_module()
    rows, d, vocab = 520, 64, 2000
    gen = torch.Generator(device="cuda").manual_seed(1)
    table = torch.randn(vocab, d, generator=gen, device="cuda").to(BF16)
    bias = torch.rand(d, generator=gen, device="cuda") * 4
    gate = torch.randn(rows, d, generator=gen, device="cuda").to(BF16)
    tokens, taken = (torch.randint(0, vocab, (rows,), generator=gen, device="cuda") for _ in range(2))
    adv = torch.randn(rows, generator=gen, device="cuda")

    def step():
        x, h = torch.empty(rows, d, dtype=BF16, device="cuda"), torch.empty(rows, d, dtype=BF16, device="cuda")
        fp.fsdp_embedding_forward(tokens, table, x)
        states = torch.empty(fp.fsdp_gated_scan_states(rows, d), d, device="cuda")
        fp.fsdp_gated_scan_forward(x, gate, h, bias=bias, seq_len=260, states=states)
        logits = h @ table.T
        out = [torch.empty(rows, device="cuda") for _ in range(3)]
        fp.fsdp_policy_loss_forward(logits, taken, None, adv, *out, dlogits=logits)
        dtable = logits.T @ h
        dh, dx, dgate, dbias = logits @ table, torch.empty_like(x), torch.empty_like(x), torch.empty_like(bias)
        fp.fsdp_gated_scan_backward(dh, x, gate, states, dx, dgate, bias=bias, dbias=dbias, seq_len=260)
        fp.fsdp_embedding_backward(tokens, dx, dtable, accumulate=True)
        return [out[0], dtable, dgate, dbias]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for seed in (2, 3):
        tokens.copy_(torch.randint(0, vocab, (rows,), device="cuda"))
        adv.normal_()
        graph.replay()
        want = step()
        assert all(torch.equal(a, b) for a, b in zip(held, want))
    fp.fsdp_ops_sync_status()

"""Embedding lookup and its gradient against their definitions in 64 bits.

Tolerances, in units u = 2^-24.  A looked-up value is one product and one rounding.  A token's n rows are summed by chains
that come to at most n + 16 additions, so a sum is off by at most (n + 16) u times the sum of magnitudes; scaling, adding the old
value and rounding to the result's type add a rounding each."""
import threading

import pytest
import torch

from gpu_util import fp_module
from ops_util import BF16, EPS32, F32, F64, HALF, Matrix, close, normals

pytestmark = pytest.mark.gpu


def tokens_of(seed, rows, vocab, kind="skewed"):
    gen = torch.Generator().manual_seed(seed)
    if kind == "one":
        return torch.full((rows,), vocab // 2)
    if kind == "distinct":
        return torch.randperm(vocab, generator=gen)[:rows]
    t = (torch.rand(rows, generator=gen, dtype=F64) * torch.log(torch.tensor(float(vocab + 1)))).exp().long() - 1
    t = torch.randperm(vocab, generator=gen)[t.clamp(0, vocab - 1)]
    return torch.where(torch.rand(rows, generator=gen) < 0.05, torch.randint(-3, 0, (rows,), generator=gen), t)


def check_forward(fp, tokens, vocab, cols, w_dtype, o_dtype, index=torch.int64, ld=None, offset=0, scale=32.0):
    rows = tokens.numel()
    weight = normals(vocab + cols, vocab, cols).to(w_dtype)
    mw = Matrix(vocab, cols, w_dtype, ld, offset, weight)
    mo = Matrix(rows, cols, o_dtype, ld, offset)
    fp.fsdp_embedding_forward(tokens.to(index).cuda(), mw.t, mo.t, scale=scale)
    good = (tokens >= 0) & (tokens < vocab)
    want = torch.where(good[:, None], weight.double()[tokens.clamp(0, vocab - 1)] * scale, 0.0)
    close(mo.t, want, want.abs() * (HALF[o_dtype] + EPS32) + 1e-40, "out")
    assert mo.intact() and mw.intact()


def check_backward(fp, tokens, vocab, cols, g_dtype, d_dtype, add=False, index=torch.int64, ld=None, offset=0, scale=0.5, seed=0):
    rows = tokens.numel()
    dout = normals(seed + 1, rows, cols).to(d_dtype)
    old = normals(seed + 2, vocab, cols).to(g_dtype)
    md = Matrix(rows, cols, d_dtype, ld, offset, dout)
    mg = Matrix(vocab, cols, g_dtype, ld, offset, old if add else None)
    fp.fsdp_embedding_backward(tokens.to(index).cuda(), md.t, mg.t, scale=scale, accumulate=add)
    good = (tokens >= 0) & (tokens < vocab)
    want, size, n = torch.zeros(vocab, cols, dtype=F64), torch.zeros(vocab, cols, dtype=F64), torch.zeros(vocab, dtype=F64)
    want.index_add_(0, tokens[good], dout.double()[good] * scale)
    size.index_add_(0, tokens[good], dout.double()[good].abs() * scale)
    n.index_add_(0, tokens[good], torch.ones(int(good.sum()), dtype=F64))
    tol = (n[:, None] + 16) * EPS32 * size
    if add:
        want += old.double()
        tol += EPS32 * want.abs()
    close(mg.t, want, tol + (want.abs() + tol) * HALF[g_dtype], "dweight")
    if add:  # rows without tokens keep their bits
        assert torch.equal(mg.t.cpu()[n == 0], old[n == 0])
    assert mg.intact() and md.intact()


WIDTHS = [1, 7, 8, 64, 72, 255, 256, 515, 1024, 1409, 2056]


@pytest.mark.parametrize("w_dtype,o_dtype", [(BF16, BF16), (F32, F32), (F32, BF16), (BF16, F32)])
@pytest.mark.parametrize("cols", WIDTHS)
def test_forward(cols, w_dtype, o_dtype):
    check_forward(fp_module(), tokens_of(cols, 37, 50), 50, cols, w_dtype, o_dtype)


@pytest.mark.parametrize("g_dtype,d_dtype", [(BF16, BF16), (F32, F32), (F32, BF16), (BF16, F32)])
@pytest.mark.parametrize("cols", WIDTHS)
def test_backward(cols, g_dtype, d_dtype):
    check_backward(fp_module(), tokens_of(cols, 237, 90), 90, cols, g_dtype, d_dtype)
    check_backward(fp_module(), tokens_of(cols, 237, 90), 90, cols, g_dtype, d_dtype, add=True)


@pytest.mark.parametrize("rows", [0, 1, 2, 7, 8, 9, 31, 4095, 4096, 4097, 8193, 30011])
@pytest.mark.parametrize("vocab", [1, 2, 3, 1000, 1023, 1024, 70001])
def test_backward_sizes(rows, vocab):
    fp = fp_module()
    for add in (False, True):
        check_backward(fp, tokens_of(rows, rows, vocab), vocab, 24, F32, BF16, add=add, index=torch.int32)


@pytest.mark.parametrize("rows", [5, 300, 5000, 20011])
@pytest.mark.parametrize("kind", ["one", "distinct"])
def test_backward_frequencies(rows, kind):
    check_backward(fp_module(), tokens_of(rows, rows, 30000, kind), 30000, 40, BF16, BF16)
    check_backward(fp_module(), tokens_of(rows, rows, 30000, kind), 30000, 33, F32, F32, add=True)


def test_backward_of_a_large_vocabulary():
    """Three sorting passes: keys of more than 20 bits."""
    check_backward(fp_module(), tokens_of(3, 9001, 1_200_007), 1_200_007, 8, BF16, BF16)


def test_backward_of_many_rows():
    """Several blocks of counts, long pieces, and one token that fills many of them."""
    t = tokens_of(4, 300_007, 5000)
    t[::2] = 77
    check_backward(fp_module(), t, 5000, 16, F32, BF16)


@pytest.mark.parametrize("ld,offset", [(64, 1), (72, 0), (65, 0), (64, 8), (66, 3)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_strides(ld, offset, dtype):
    fp = fp_module()
    t = tokens_of(ld, 130, 40)
    check_forward(fp, t, 40, 64, dtype, dtype, ld=ld, offset=offset)
    check_backward(fp, t, 40, 64, dtype, dtype, ld=ld, offset=offset)
    check_backward(fp, t, 40, 64, dtype, dtype, add=True, ld=ld, offset=offset)


@pytest.mark.parametrize("index", [torch.int32, torch.int64])
def test_tokens_outside_the_vocabulary(index):
    """The values next to the borders, the type's extremes and, in 64 bits, values whose low half would be a token."""
    fp = fp_module()
    low = torch.iinfo(index)
    odd = [-1, 40, 41, low.min, low.max] + ([1 << 32, (1 << 32) + 3, -(1 << 32)] if index == torch.int64 else [])
    t = torch.tensor([0, 39] + odd + [39, 5])
    check_forward(fp, t, 40, 48, BF16, BF16, index=index)
    check_backward(fp, t, 40, 48, F32, BF16, index=index)
    check_backward(fp, torch.tensor(odd), 40, 48, F32, BF16, index=index)
    check_backward(fp, torch.tensor(odd), 40, 48, BF16, BF16, index=index, add=True)


def test_specials_stay_with_their_token():
    """A NaN or an infinity reaches the rows of its own token, and nothing through a scale of 0 times a missing row."""
    fp = fp_module()
    t = torch.tensor([3, 5, -1, 3, 7])
    dout = torch.ones(5, 16)
    dout[1, 2], dout[2, 4], dout[3, 6] = float("nan"), float("nan"), float("inf")
    g = torch.empty(9, 16, device="cuda")
    fp.fsdp_embedding_backward(t.cuda(), dout.cuda(), g)
    want = torch.zeros(9, 16)
    want[3], want[5], want[7] = 2.0, 1.0, 1.0
    want[5, 2], want[3, 6] = float("nan"), float("inf")
    assert torch.equal(torch.nan_to_num(g.cpu(), 77.0, 88.0), torch.nan_to_num(want, 77.0, 88.0))
    out = torch.empty(5, 16, device="cuda")
    fp.fsdp_embedding_forward(t.cuda(), torch.full((9, 16), float("inf"), device="cuda"), out)
    assert bool((out[2] == 0).all()) and bool(torch.isinf(out[[0, 1, 3, 4]]).all())


def test_gradient_is_the_lookups_derivative():
    """<dout, forward(w + e v) - forward(w)> = e <backward(dout), v> for this linear operator, with values whose sums are exact."""
    fp = fp_module()
    gen = torch.Generator().manual_seed(2)
    t = tokens_of(9, 600, 64).cuda()
    w, v = (torch.randint(-8, 9, (64, 40), generator=gen).float().cuda() for _ in range(2))
    dout = torch.randint(-8, 9, (600, 40), generator=gen).float().cuda()
    a, b, g = torch.empty_like(dout), torch.empty_like(dout), torch.empty_like(w)
    fp.fsdp_embedding_forward(t, w, a, scale=2.0)
    fp.fsdp_embedding_forward(t, w + v, b, scale=2.0)
    fp.fsdp_embedding_backward(t, dout, g, scale=2.0)
    assert float((dout.double() * (b - a).double()).sum()) == float((g.double() * v.double()).sum())


def test_same_bits_streams_graphs_and_threads():
    fp = fp_module()
    t = tokens_of(1, 9000, 700).cuda()
    dout = torch.randn(9000, 136, device="cuda").to(BF16)
    first = torch.empty(700, 136, dtype=BF16, device="cuda")
    fp.fsdp_embedding_backward(t, dout, first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = torch.empty_like(first)
    fp.fsdp_embedding_backward(t, dout, other, stream=side)
    side.synchronize()
    assert torch.equal(first, other)
    # Captured, replayed on other tokens.
    ws = torch.empty(fp.fsdp_embedding_workspace(9000, 700, 136), dtype=torch.uint8, device="cuda")
    graph, held, out = torch.cuda.CUDAGraph(), t.clone(), torch.empty_like(first)
    with torch.cuda.graph(graph):
        fp.fsdp_embedding_backward(held, dout, out, workspace=ws)
    for seed in (5, 6):
        held.copy_(tokens_of(seed, 9000, 700))
        ws.fill_(0xFF)
        graph.replay()
        fp.fsdp_embedding_backward(held, dout, other)
        assert torch.equal(out, other)
    # Two threads on streams of their own.
    got = [torch.empty_like(first) for _ in range(2)]

    def go(k):
        s = torch.cuda.Stream()
        for _ in range(20):
            fp.fsdp_embedding_backward(t, dout, got[k], stream=s)
        s.synchronize()

    torch.cuda.synchronize()
    threads = [threading.Thread(target=go, args=(k,)) for k in range(2)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert torch.equal(got[0], first) and torch.equal(got[1], first)


def test_binding_refusals():
    fp = fp_module()
    w, out, t = torch.empty(9, 16, device="cuda"), torch.empty(4, 16, device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda")
    bad = [((t.float(), w, out), "not one of"), ((t.cpu(), w, out), "CUDA"), ((t, w, out[:3]), "not 4"), ((t, w.half(), out), "float16"),
           ((t, w, torch.empty(4, 15, device="cuda")), "not 4 x 16"), ((t.repeat(2)[::2], w, out), "contiguous"), ((t, w[0], out), "dimensions"),
           (([0], w, out), "not a tensor")]
    for args, word in bad:
        with pytest.raises(ValueError, match=word):
            fp.fsdp_embedding_forward(*args)
    with pytest.raises(ValueError, match="workspace holds"):
        fp.fsdp_embedding_backward(t, out, w, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    with pytest.raises(fp.FsdpError, match="scale"):
        fp.fsdp_embedding_forward(t, w, out, scale=float("nan"))

"""The training operators on matrices of more than 2^31 elements, whose last rows are compared with the same rows computed
alone; and waits that give up."""
import contextlib
from concurrent.futures import ThreadPoolExecutor

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


def test_act8_beyond_32_bits():
    fp = fp_module()
    rows, cols = 70001, 32768
    x = rows_of(rows, cols, 1)
    kept = fp.Act8(rows, cols)
    fp.fsdp_act8_store(x, kept)
    y = torch.empty_like(x)
    fp.fsdp_act8_load(kept, y)
    last = fp.Act8(7, cols)
    fp.fsdp_act8_store(x[-7:], last)
    z = torch.empty(7, cols, dtype=BF16, device="cuda")
    fp.fsdp_act8_load(last, z)
    assert torch.equal(y[-7:], z) and torch.equal(y[:7], y[1031:1038])


def test_act8_rows_far_apart():
    """Rows that are far apart and off a vector's boundary: offsets pass 2^32 bytes element by element too."""
    fp = fp_module()
    flat = torch.zeros(5 * (1 << 30), dtype=torch.uint8, device="cuda").view(BF16)
    x = flat[:(1 << 30) * 2].view(2, 1 << 30)[:, 1:100]
    x.copy_(torch.randn(2, 99))
    kept = fp.Act8(2, 99)
    fp.fsdp_act8_store(x, kept)
    y = torch.empty(2, 99, device="cuda")
    fp.fsdp_act8_load(kept, y)
    same = fp.Act8(2, 99)
    fp.fsdp_act8_store(x.contiguous(), same)
    assert torch.equal(kept.data, same.data) and bool(((y - x.float()).abs() <= x.float().abs().amax() / 63).all())


@pytest.mark.parametrize("cols", [32768, 32767])
def test_norm_beyond_32_bits(cols):
    fp = fp_module()
    rows = 66001
    x, dy = rows_of(rows, cols, 2), rows_of(rows, cols, 3, std=0.1)
    w, b = torch.rand(cols, device="cuda") + 0.5, torch.rand(cols, device="cuda")

    def both(x, dy):
        n = x.shape[0]
        y, dx = torch.empty_like(x), torch.empty_like(x)
        mean, rstd = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
        fp.fsdp_layer_norm_forward(x, w, b, y, mean, rstd)
        dw = torch.empty(cols, device="cuda")
        fp.fsdp_layer_norm_backward(dy, x, w, mean, rstd, dx, dw)
        return y, mean, rstd, dx

    whole, last = both(x, dy), both(x[-7:], dy[-7:])
    fp.fsdp_ops_sync_status()
    for p, q in zip(whole, last):
        assert torch.equal(p[-7:], q)


def test_ffn_beyond_32_bits():
    fp = fp_module()
    rows, d, f = 1_060_003, 64, 2056
    x = rows_of(rows, d, 4)
    wg, wu = (rows_of(f, d, s, std=0.125) for s in (5, 6))
    h = torch.empty(rows, f, dtype=BF16, device="cuda")
    gate, up = fp.Act8(rows, f), fp.Act8(rows, f)
    fp.fsdp_gated_ffn_forward(x, wg, wu, h, gate=gate, up=up)
    # The last whole tile on its own.
    n = rows % 256 or 256
    hl, gl, ul = torch.empty(n, f, dtype=BF16, device="cuda"), fp.Act8(n, f), fp.Act8(n, f)
    fp.fsdp_gated_ffn_forward(x[-n:], wg, wu, hl, gate=gl, up=ul)
    assert torch.equal(h[-n:], hl)
    y, z = torch.empty_like(h), torch.empty_like(hl)
    fp.fsdp_act8_load(up, y)
    fp.fsdp_act8_load(ul, z)
    assert torch.equal(y[-n:], z)
    del y
    dh = rows_of(rows, f, 7, std=0.01)
    dx, dxl = torch.empty_like(x), torch.empty(n, d, dtype=BF16, device="cuda")
    dwg, dwu = torch.empty_like(wg), torch.empty_like(wu)
    fp.fsdp_gated_ffn_backward(dh, x, wg, wu, dx, dwg, dwu, gate=gate, up=up)
    fp.fsdp_gated_ffn_backward(dh[-n:], x[-n:], wg, wu, dxl, gate=gl, up=ul)
    fp.fsdp_ops_sync_status()
    # Another split of the K loop may round a sum the other way.
    assert bool(((dx[-n:] - dxl).abs().float() <= dxl.abs().float() * 2 ** -7 + 1e-4).all())
    assert bool(torch.isfinite(dwg).all()) and bool(torch.isfinite(dwu).all())


def test_norm_wait_that_gives_up():
    fp = fp_module()
    x = torch.randn(3000, 1024, device="cuda")
    y = torch.empty_like(x)
    fp.fsdp_layer_norm_forward(x, None, None, y)
    mean, rstd = torch.zeros(3000, device="cuda"), torch.ones(3000, device="cuda")
    dx, dw = torch.empty_like(x), torch.empty(1024, device="cuda")
    fp.fsdp_layer_norm_backward(x, x, None, mean, rstd, dx, dw)
    fp.fsdp_ops_sync_status()
    fp.fsdp_debug_set_wait_fault(1, 20_000_000)
    try:
        z = torch.empty_like(x)
        fp.fsdp_layer_norm_forward(x, None, None, z)
        with pytest.raises(fp.FsdpError, match="gave up"):
            fp.fsdp_ops_sync_status()
        fp.fsdp_layer_norm_backward(x, x, None, mean, rstd, torch.empty_like(x), torch.empty_like(dw))
        with pytest.raises(fp.FsdpError, match="gave up"):
            fp.fsdp_ops_sync_status()
    finally:
        fp.fsdp_debug_set_wait_fault(0, 0)
    again, dxa, dwa = torch.empty_like(x), torch.empty_like(dx), torch.empty_like(dw)
    fp.fsdp_layer_norm_forward(x, None, None, again)
    fp.fsdp_layer_norm_backward(x, x, None, mean, rstd, dxa, dwa)
    fp.fsdp_ops_sync_status()
    assert torch.equal(again, y) and torch.equal(dxa, dx) and torch.equal(dwa, dw)


@pytest.mark.parametrize("cols,group", [(1024, 23), (1024, 5), (4096, 5), (2048, 1)])
def test_norm_wait_that_gives_up_in_a_later_group(cols, group):
    """A row group of a block gives up long after the first one has left: the status says so all the same.  One row to
    each group of every SM (24 groups of a block up to 1,024 columns, 6 to 4,096), so that the first block has them all."""
    fp = fp_module()
    groups = 24 if cols <= 1024 else 6
    x = torch.randn(torch.cuda.get_device_properties(0).multi_processor_count * groups, cols, device="cuda")
    y = torch.empty_like(x)
    fp.fsdp_layer_norm_forward(x, None, None, y)
    fp.fsdp_ops_sync_status()
    fp.fsdp_debug_set_wait_fault(1 + 256 * group, 20_000_000)
    try:
        fp.fsdp_layer_norm_forward(x, None, None, torch.empty_like(x))
        with pytest.raises(fp.FsdpError, match="gave up"):
            fp.fsdp_ops_sync_status()
    finally:
        fp.fsdp_debug_set_wait_fault(0, 0)
    again = torch.empty_like(x)
    fp.fsdp_layer_norm_forward(x, None, None, again)
    fp.fsdp_ops_sync_status()
    assert torch.equal(again, y)


@pytest.mark.parametrize("group", [1, 7])
def test_norm_backward_wait_that_gives_up_in_a_later_group(group):
    """The same of the backward pass, eight groups of a block to 1,024 columns."""
    fp = fp_module()
    x = torch.randn(torch.cuda.get_device_properties(0).multi_processor_count * 8, 1024, device="cuda")
    mean, rstd = torch.zeros(x.shape[0], device="cuda"), torch.ones(x.shape[0], device="cuda")
    fp.fsdp_ops_sync_status()
    fp.fsdp_debug_set_wait_fault(1 + 256 * group, 20_000_000)
    try:
        fp.fsdp_layer_norm_backward(x, x, None, mean, rstd, torch.empty_like(x), torch.empty(1024, device="cuda"))
        with pytest.raises(fp.FsdpError, match="gave up"):
            fp.fsdp_ops_sync_status()
    finally:
        fp.fsdp_debug_set_wait_fault(0, 0)
    fp.fsdp_ops_sync_status()


def test_every_thread_is_told_of_a_wait_that_gave_up():
    """One thread's asking does not take the failure away from another, whose results it may be."""
    fp = fp_module()
    x = torch.randn(300, 1024, device="cuda")

    def told():
        try:
            fp.fsdp_ops_sync_status()
        except fp.FsdpError as e:
            assert e.status == fp.FSDP_ETIMEOUT and "gave up" in str(e)
            return True
        return False

    def forward():
        y = torch.empty_like(x)
        fp.fsdp_layer_norm_forward(x, None, None, y)
        torch.cuda.synchronize()

    with contextlib.ExitStack() as stack:
        one, two = (stack.enter_context(ThreadPoolExecutor(1)) for _ in range(2))
        threads = [lambda f: f(), lambda f: one.submit(f).result(), lambda f: two.submit(f).result()]
        forward()
        for run in threads:
            run(told)  # earlier failures, of which a new thread is told too
        assert not any(run(told) for run in threads)
        fp.fsdp_debug_set_wait_fault(1, 20_000_000)
        try:
            two.submit(forward).result()
        finally:
            fp.fsdp_debug_set_wait_fault(0, 0)
        assert [run(told) for run in threads] == [True, True, True]
        forward()
        assert not any(run(told) for run in threads)

"""The example's block: its gradients against the formulas in 64 bits, and steps that lower the loss."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("ffn_block_step", os.path.join(ROOT, "examples", "ffn_block_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_gradients(example):
    """One step's packed gradients.  8-bit gate, up and input each carry an error of about 0.8 % of their spread, BF16
    operands 0.2 %; the errors are independent from element to element, so a gradient that sums over 512 tokens is within
    2 % in the 2-norm."""
    block = example.Block(96, 200, 3)
    gen = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(512, 96, generator=gen, device="cuda").to(torch.bfloat16)
    target = torch.randn(512, 96, generator=gen, device="cuda")
    params = [p.double().requires_grad_() for p in block.params]
    loss = block.step(x, target, 0.0)
    w, b, gate, up, down = params
    y = torch.nn.functional.layer_norm(x.double(), (96,), w, b, 1e-5)
    out = x.double() + (torch.nn.functional.silu(y @ gate.T) * (y @ up.T)) @ down.T
    want = (out - target).square().mean()
    assert abs(float(loss) - float(want.detach())) <= 2e-2 * float(want.detach())
    for got, ref in zip(block.sharded, torch.autograd.grad(want, params)):
        ref = ref.reshape(-1)
        assert float((got - ref).norm()) <= 2e-2 * float(ref.norm())


def test_learns(example):
    losses = example.train(steps=30, tokens=1000, d=128, f=320)
    assert losses[-1] < 0.6 * losses[0]

"""The recurrent example: its gradients against the formulas in 64 bits, its steps, and generation against the whole pass."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("recurrent_model_step", os.path.join(ROOT, "examples", "recurrent_model_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def reference(model, params, tokens, offsets):
    """Logits in 64 bits from the parameters' values."""
    table, weight, bias, w_in, w_gate, gate_bias, w_out = params
    x = table[tokens] * model.scale
    y = torch.nn.functional.layer_norm(x, (model.d,), weight, bias, 1e-5)
    u, a = y @ w_in.T, torch.sigmoid(y @ w_gate.T + gate_bias)
    h = []
    off = offsets.tolist()
    for lo, hi in zip(off, off[1:]):
        state = torch.zeros(model.d, dtype=torch.float64, device="cuda")
        for t in range(lo, hi):
            state = a[t] * state + (1 - a[t]) * u[t]
            h.append(state)
    return (x + torch.stack(h) @ w_out.T) @ table.T


@pytest.mark.parametrize("loss", ["distill", "policy"])
def test_gradients(example, loss):
    """One step's packed gradients.  Between the formulas and the step lie BF16 activations and gradients (each rounding 2^-9 of
    its value in the mean), some ten of them in a row, and the norm's 8-bit checkpoint (0.8 % of its input's spread in the norm's
    own gradient); errors are independent from element to element, so a gradient that sums over 500 tokens is within 3 % in
    the 2-norm."""
    d, vocab, n, top = 72, 300, 500, 9
    model = example.Model(vocab, d, 3)
    tokens, offsets, weight = example.batch(n, vocab, 4)
    gen = torch.Generator(device="cuda").manual_seed(5)
    ids = torch.stack([torch.randperm(vocab, generator=gen, device="cuda")[:top] for _ in range(n)])
    teacher = torch.randn(n, top, generator=gen, device="cuda")
    taken, adv = ids[:, 0].contiguous(), torch.randn(n, generator=gen, device="cuda")
    params = [p.double().requires_grad_() for p in model.params]
    logp = torch.log_softmax(reference(model, params, tokens, offsets), -1)
    if loss == "distill":
        q = torch.softmax(teacher.double(), -1)
        rows = (q * (torch.log(q) - logp.gather(1, ids))).sum(-1)
        loss_of = example.distill_loss(ids, teacher, weight)
    else:
        # Ratios that BF16 logits cannot move across a border: half of them near 1, the others far outside.
        lp = logp.gather(1, taken[:, None])[:, 0]
        old = (lp.detach() + torch.where(torch.arange(n, device="cuda") % 2 == 0, 0.02, 0.7)).float()
        r, gap = torch.exp(lp - old.double()), (old - 0.1).double() - lp
        rows = -torch.minimum(r * adv, r.clip(0.8, 1.2) * adv) + 0.05 * (torch.exp(gap) - gap - 1)
        loss_of = example.policy_loss(taken, old, adv, old - 0.1, weight)
    want = (rows * weight.double()).sum()
    got = model.step(tokens, offsets, loss_of, 0.0)
    assert abs(float(got) - float(want.detach())) <= 2e-2 * float((rows * weight.double()).abs().sum().detach())
    for g, ref in zip(model.sharded, torch.autograd.grad(want, params)):
        ref = ref.reshape(-1)
        assert float((g - ref).norm()) <= 3e-2 * float(ref.norm())


@pytest.mark.parametrize("loss", ["distill", "policy"])
def test_runs(example, loss):
    losses = example.train(steps=3, tokens=1000, d=128, vocab=1000, loss=loss)
    assert len(losses) == 3 and all(abs(v) < 1e3 for v in losses)


def test_generation_follows_the_whole_pass(example):
    """Token by token, each sequence's logits are those of the pass over the whole batch, to BF16's roundings."""
    model = example.Model(500, 64, 7)
    tokens = torch.randint(0, 500, (4, 12), device="cuda")
    whole, _ = model.forward(tokens.reshape(-1), torch.arange(5, device="cuda") * 12)
    states = torch.zeros(4, 64, device="cuda")
    for t in range(12):
        logits = model.generate(tokens[:, t].contiguous(), states)
        want = whole.view(4, 12, -1)[:, t].float()
        assert float((logits.float() - want).norm()) <= 1e-2 * float(want.norm())

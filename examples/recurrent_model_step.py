"""Training steps of a small recurrent language model whose parameters form one fully_shard group.

One layer, ``x + out(scan(in(norm(x)), gate(norm(x))))``, between an embedding and an output layer that share their table.  The
group mixes dtypes as such layers do: BF16 matrices, an FP32 norm and an FP32 gate bias per channel.  One step, on one GPU (world
size 1, where the packed buffers are their own reduce-scatter and all-gather results):

  forward    the scaled lookup; layer norm, which keeps the 8-bit checkpoint of its input; the gated recurrence over packed
             sequences, which keeps its states some rows apart; logits; the loss and, in the same pass and the same
             memory, its gradient: distillation from a teacher's top logits, or the clipped policy loss
  backward   the output layer's gradient; the recurrence's, with the gate bias's; the norm's from its checkpoint; the
             embedding's, added to the output layer's in the shared table
  exchange   the gradients, FP32 and BF16, packed into one FP32 bucket; an SGD step on the FP32 shards; the shards packed,
             cast and unpacked into the compute parameters

``Model.generate`` is the same model token by token, with one state per sequence.

Run: python examples/recurrent_model_step.py [--steps 20] [--tokens 4096] [--d 512] [--vocab 8192] [--loss distill]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from fsdp2_gradient_packing_gb300 import fsdp_pack as fp  # noqa: E402

F32, BF16 = fp.FSDP_DTYPE_F32, fp.FSDP_DTYPE_BF16


class Model:
    """Parameters as one group: FP32 shards, compute parameters and gradients in the policy's dtypes."""

    def __init__(self, vocab, d, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.vocab, self.d, self.scale = vocab, d, 2.0
        shapes = {"table": (vocab, d), "norm_weight": (d,), "norm_bias": (d,), "w_in": (d, d), "w_gate": (d, d), "gate_bias": (d,),
                  "w_out": (d, d)}

        def normal(name):
            return torch.randn(*shapes[name], generator=gen, device="cuda") * d ** -0.5

        shards = [normal("table"), torch.ones(d, device="cuda"), torch.zeros(d, device="cuda"), normal("w_in"), normal("w_gate"),
                  torch.linspace(0, 5, d, device="cuda"), normal("w_out")]
        self.shards = [s.reshape(-1) for s in shards]
        kinds = [F32 if len(s) == 1 else BF16 for s in shapes.values()]  # gradient and compute dtype of each parameter
        self.layout = fp.fsdp_plan_layout([(s.numel(), k, F32, F32, k) for s, k in zip(self.shards, kinds)], 1)
        info = fp.fsdp_layout_query(self.layout)
        dtype = {F32: torch.float32, BF16: torch.bfloat16}
        self.params = [torch.empty(s, dtype=dtype[k], device="cuda") for s, k in zip(shapes.values(), kinds)]
        self.grads = [torch.empty_like(p) for p in self.params]
        self.bucket = torch.empty(info.total_numel, device="cuda")
        self.gathered = torch.empty(info.ag_bytes, dtype=torch.uint8, device="cuda")
        self.sharded = [torch.empty_like(s) for s in self.shards]
        self.unshard()

    def unshard(self):
        fp.fsdp_allgather_copy_in(self.layout, self.shards, self.gathered)
        fp.fsdp_allgather_copy_out(self.layout, self.gathered, self.params)

    def forward(self, tokens, offsets):
        """Logits, and what the backward pass needs."""
        table, weight, bias, w_in, w_gate, gate_bias, _ = self.params
        rows, d = tokens.numel(), self.d
        x = torch.empty(rows, d, dtype=torch.bfloat16, device="cuda")
        fp.fsdp_embedding_forward(tokens, table, x, scale=self.scale)
        y, mean, rstd, kept = torch.empty_like(x), torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda"), fp.Act8(rows, d)
        fp.fsdp_layer_norm_forward(x, weight, bias, y, mean, rstd, keep=kept)
        u, g, h = y @ w_in.T, y @ w_gate.T, torch.empty_like(x)
        states = torch.empty(fp.fsdp_gated_scan_states(rows, d), d, device="cuda")
        fp.fsdp_gated_scan_forward(u, g, h, bias=gate_bias, offsets=offsets, states=states)
        top = x + h @ self.params[6].T
        return top @ table.T, (kept, mean, rstd, y, u, g, h, states, top)

    def backward(self, tokens, offsets, dlogits, saved):
        """Gradients of all parameters into ``grads``."""
        table, weight, _, w_in, w_gate, gate_bias, w_out = self.params
        dtable, dweight, dbias, dw_in, dw_gate, dgate_bias, dw_out = self.grads
        kept, mean, rstd, y, u, g, h, states, top = saved
        torch.mm(dlogits.T, top, out=dtable)
        dtop = dlogits @ table
        torch.mm(dtop.T, h, out=dw_out)
        dh, du, dg = dtop @ w_out, torch.empty_like(u), torch.empty_like(g)
        fp.fsdp_gated_scan_backward(dh, u, g, states, du, dg, bias=gate_bias, dbias=dgate_bias, offsets=offsets)
        torch.mm(du.T, y, out=dw_in)
        torch.mm(dg.T, y, out=dw_gate)
        dy, dx = du @ w_in + dg @ w_gate, torch.empty_like(dtop)
        fp.fsdp_layer_norm_backward(dy, kept, weight, mean, rstd, dx, dweight, dbias)
        fp.fsdp_embedding_backward(tokens, dtop + dx, dtable, scale=self.scale, accumulate=True)

    def step(self, tokens, offsets, loss_of, rate):
        """One step; ``loss_of(logits)`` writes the gradient over the logits and returns the rows' losses.  Returns their
        sum before the step, as a tensor."""
        logits, saved = self.forward(tokens, offsets)
        loss = loss_of(logits).sum()
        self.backward(tokens, offsets, logits, saved)
        fp.fsdp_pack_reduce_scatter(self.layout, self.grads, [self.bucket])
        fp.fsdp_reduce_scatter_copy_out(self.layout, [self.bucket], self.sharded)
        torch._foreach_add_(self.shards, self.sharded, alpha=-rate)
        self.unshard()
        return loss

    def generate(self, tokens, states):
        """The next token's logits of every sequence, one row each; ``states`` [sequences, d] moves on in place."""
        table, weight, bias, w_in, w_gate, gate_bias, w_out = self.params
        x = torch.empty(tokens.numel(), self.d, dtype=torch.bfloat16, device="cuda")
        fp.fsdp_embedding_forward(tokens, table, x, scale=self.scale)
        y, h = torch.empty_like(x), torch.empty_like(x)
        fp.fsdp_layer_norm_forward(x, weight, bias, y)
        fp.fsdp_gated_scan_forward(y @ w_in.T, y @ w_gate.T, h, bias=gate_bias, initial=states, final=states, seq_len=1)
        return (x + h @ w_out.T) @ table.T


def distill_loss(ids, teacher, weight):
    """Distillation from a teacher's top logits; the gradient takes the logits' place."""
    def loss_of(logits):
        loss, lse = (torch.empty(logits.shape[0], device="cuda") for _ in range(2))
        fp.fsdp_distill_loss_forward(logits, ids, teacher, loss, lse, weight=weight, dlogits=logits)
        return loss
    return loss_of


def policy_loss(taken, old_logp, advantage, ref_logp, weight, kl=0.05):
    """The clipped policy loss; the gradient takes the logits' place."""
    def loss_of(logits):
        loss, logp, lse = (torch.empty(logits.shape[0], device="cuda") for _ in range(3))
        fp.fsdp_policy_loss_forward(logits, taken, old_logp, advantage, loss, logp, lse, ref_logp=ref_logp, weight=weight, kl=kl, dlogits=logits)
        return loss
    return loss_of


def batch(tokens, vocab, seed=0):
    """Tokens of uneven sequences packed one behind the other, where they begin, and weights that leave out every fourth."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    cuts = torch.sort(torch.randint(0, tokens + 1, (7,), generator=gen, device="cuda")).values
    offsets = torch.cat([cuts.new_zeros(1), cuts, cuts.new_tensor([tokens])])
    weight = torch.where(torch.arange(tokens, device="cuda") % 4 < 3, 4 / (3 * tokens), 0.0)
    return torch.randint(0, vocab, (tokens,), generator=gen, device="cuda"), offsets, weight


def train(steps, tokens, d, vocab, loss="distill", top=32):
    """Losses of a model that learns another model's predictions, or from its rewards."""
    rate = 10.0 if loss == "distill" else 1.0  # a large step takes the policy far from the one that was sampled
    teacher, model = Model(vocab, d, 2), Model(vocab, d, 1)
    ids, offsets, weight = batch(tokens, vocab)
    logits, _ = teacher.forward(ids, offsets)
    best = torch.topk(logits, top)
    if loss == "distill":
        loss_of = distill_loss(best.indices, best.values, weight)
    else:
        own, _ = model.forward(ids, offsets)
        taken = torch.multinomial(torch.softmax(own.float(), -1), 1)[:, 0]
        old = torch.log_softmax(own.float(), -1).gather(1, taken[:, None])[:, 0]
        reward = logits.float().gather(1, taken[:, None])[:, 0]
        loss_of = policy_loss(taken, old, (reward - reward.mean()) / reward.std(), old, weight)
    losses = [model.step(ids, offsets, loss_of, rate) for _ in range(steps)]
    fp.fsdp_ops_sync_status()
    fp.fsdp_sync_status(model.layout)
    return [float(v) for v in losses]


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--d", type=int, default=512)
    ap.add_argument("--vocab", type=int, default=8192)
    ap.add_argument("--loss", choices=["distill", "policy"], default="distill")
    a = ap.parse_args()
    for k, v in enumerate(train(a.steps, a.tokens, a.d, a.vocab, a.loss)):
        print(f"step {k:3d}  loss {v:.5f}")


if __name__ == "__main__":
    main()

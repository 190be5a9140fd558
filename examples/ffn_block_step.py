"""Training steps of one pre-norm gated feed-forward block whose parameters form one fully_shard group.

The block is ``x + down(act(gate(norm(x))) * up(norm(x)))`` with an FP32 layer norm and BF16 matrices, a group of mixed
dtypes.  One step, on one GPU (world size 1, where the packed buffers are their own reduce-scatter and all-gather results):

  forward    layer norm, which keeps the 8-bit checkpoint of its input; the gated feed-forward call, which keeps gate and up
             in 8 bits; the down projection, a plain product
  backward   the down projection's gradients; the norm's output computed again from the checkpoint; the feed-forward
             block's gradients from the 8-bit gate and up; the norm's from the checkpoint of its input
  exchange   the gradients, FP32 and BF16, packed into one FP32 bucket; an SGD step on the FP32 shards; the shards packed,
             cast and unpacked into the compute parameters

Run: python examples/ffn_block_step.py [--steps 20] [--tokens 4096] [--d 512] [--f 1408]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from fsdp2_gradient_packing_gb300 import fsdp_pack as fp  # noqa: E402

F32, BF16 = fp.FSDP_DTYPE_F32, fp.FSDP_DTYPE_BF16


class Block:
    """Parameters of the block as one group: FP32 shards, compute parameters and gradients in the policy's dtypes."""

    def __init__(self, d, f, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.d, self.f = d, f
        shapes = {"weight": (d,), "bias": (d,), "gate": (f, d), "up": (f, d), "down": (d, f)}
        shards = [torch.ones(d, device="cuda"), torch.zeros(d, device="cuda")]
        shards += [torch.randn(*shapes[n], generator=gen, device="cuda") * shapes[n][1] ** -0.5 for n in ("gate", "up", "down")]
        self.shards = [s.reshape(-1) for s in shards]
        kinds = [F32, F32, BF16, BF16, BF16]  # gradient and compute dtype of each parameter
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

    def step(self, x, target, rate):
        """One step on x [tokens, d] (BF16); returns the loss before it, as a tensor."""
        weight, bias, gate, up, down = self.params
        dweight, dbias, dgate, dup, ddown = self.grads
        rows, d = x.shape
        f = self.f
        y, h = torch.empty_like(x), torch.empty(rows, f, dtype=x.dtype, device=x.device)
        mean, rstd = (torch.empty(rows, device=x.device) for _ in range(2))
        kept_x, kept_gate, kept_up = fp.Act8(rows, d), fp.Act8(rows, f), fp.Act8(rows, f)
        # Forward
        fp.fsdp_layer_norm_forward(x, weight, bias, y, mean, rstd, keep=kept_x)
        fp.fsdp_gated_ffn_forward(y, gate, up, h, gate=kept_gate, up=kept_up)
        error = (x + h @ down.T).float() - target
        loss = error.square().mean()
        del y
        # Backward
        dout = (error * (2 / error.numel())).to(x.dtype)
        torch.mm(dout.T, h, out=ddown)
        dh = dout @ down
        y, dy, dx = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
        fp.fsdp_layer_norm_forward(kept_x, weight, bias, y)
        fp.fsdp_gated_ffn_backward(dh, y, gate, up, dy, dgate, dup, gate=kept_gate, up=kept_up)
        fp.fsdp_layer_norm_backward(dy, kept_x, weight, mean, rstd, dx, dweight, dbias)
        dx += dout  # what the block below would receive
        # Exchange and update
        fp.fsdp_pack_reduce_scatter(self.layout, self.grads, [self.bucket])
        fp.fsdp_reduce_scatter_copy_out(self.layout, [self.bucket], self.sharded)
        torch._foreach_add_(self.shards, self.sharded, alpha=-rate)
        self.unshard()
        return loss


def train(steps, tokens, d, f, rate=20.0, seed=0):
    """Losses of a block that learns another block's outputs."""
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    teacher, block = Block(d, f, seed + 2), Block(d, f, seed)
    x = torch.randn(tokens, d, generator=gen, device="cuda").to(torch.bfloat16)
    weight, bias, gate, up, down = teacher.params
    y, h = torch.empty_like(x), torch.empty(tokens, f, dtype=x.dtype, device="cuda")
    fp.fsdp_layer_norm_forward(x, weight, bias, y)
    fp.fsdp_gated_ffn_forward(y, gate, up, h)
    target = (x + h @ down.T).float()
    losses = [block.step(x, target, rate) for _ in range(steps)]
    fp.fsdp_ops_sync_status()
    fp.fsdp_sync_status(block.layout)
    return [float(v) for v in losses]


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--d", type=int, default=512)
    ap.add_argument("--f", type=int, default=1408)
    a = ap.parse_args()
    losses = train(a.steps, a.tokens, a.d, a.f)
    kept = fp.fsdp_act8_bytes(a.tokens, a.d) + 2 * fp.fsdp_act8_bytes(a.tokens, a.f)
    print(f"kept for the backward pass: {kept / 2 ** 20:.1f} MiB in 8 bits "
          f"({2 * a.tokens * (a.d + 2 * a.f) / 2 ** 20:.1f} MiB in BF16)")
    for k, v in enumerate(losses):
        print(f"step {k:3d}  loss {v:.5f}")


if __name__ == "__main__":
    main()

"""Train one feed-forward layer on one GPU with blockwise-FP8 weights: the layer's forward and backward
run on the FP8 codes and scales that the ZeRO-1 shard step writes, and its weight
gradients go straight into that step.

    python examples/train_ffn_layer.py [--steps 40] [--experts 4] [--width 512] [--inner 256]

The layer:  z0, x = norm_join(none, tokens)            (norm before the block)
            y     = feed_forward(x)                    (per expert, gated)
            z     = tokens + 0.5 gate norm(y)          (norm after it, gate and residual)
trained to reproduce, on one batch of tokens, a fixed teacher of the same form.  Everything is synthetic.  The norm weights and
the gate are plain float32 and take a plain gradient step; the three expert weights are FP32
masters in the shard, seen by the layer only as FP8 codes with one scale per 128x128 block.
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))


class Layer:
    """One layer whose expert weights live in a shard (data-parallel size 1)."""

    def __init__(self, n_experts: int, width: int, inner: int, hp, seed: int):
        import torch

        import blockwise_fp8_zero_fold_amd as fz
        from blockwise_fp8_zero_fold_amd.shard import Shard

        g = torch.Generator(device="cuda").manual_seed(seed)
        E, D, F = n_experts, width, inner
        self.n_experts, self.hp = E, hp
        self.shapes = [(E, F, D), (E, F, D), (E, D, F)]
        masters = [torch.randn(*s, device="cuda", generator=g) * s[2] ** -0.5 for s in self.shapes]
        self.shard = Shard(self.shapes, 1, 0)
        self.shard.init(hp, masters)
        self.codes = [torch.zeros(s, dtype=torch.uint8, device="cuda") for s in self.shapes]
        self.scales = [torch.zeros(s[0], -(-s[1] // 128), -(-s[2] // 128), device="cuda") for s in self.shapes]
        self.grads = [torch.zeros(s, device="cuda") for s in self.shapes]
        self.w_pre, self.w_post = torch.ones(D, device="cuda"), torch.ones(D, device="cuda")
        self.gate = torch.ones(D, device="cuda")
        # codes and scales of the untouched masters: one step that changes nothing
        rest = fz.Hparams(0.0, 0.9, 0.95, 1e-8, 0.0, 0.0, 0, 1.0, 2.0, 0.5, 1000, 0, 0, 0.0, None)
        self.shard.step(rest, self.grads, self.codes, self.scales, fold_on_read=True)
        fz.fp8z1_state_init(hp, self.shard.state)

    @property
    def weights(self):
        return list(zip(self.codes, self.scales))

    def forward(self, tokens, offsets):
        """z, and what the backward pass needs."""
        from blockwise_fp8_zero_fold_amd import block

        _, x = block.norm_join(None, tokens, w_pre=self.w_pre, dtype=tokens.dtype)
        y, (h, u, _) = block.ffn_forward(x, *self.weights, offsets=offsets, save=True)
        z, _ = block.norm_join(y, tokens, w_post=self.w_post, gate=self.gate, block_scale=0.5)
        return z, (x, y, h, u)

    def backward(self, dz, tokens, offsets, kept):
        """Fills self.grads (row-major FP32, what the shard step reads); returns the gradient at the
        tokens and those of the norm weights and the gate."""
        from blockwise_fp8_zero_fold_amd import block

        x, y, h, u = kept
        after = block.norm_join_backward(dz, None, y, dz, w_post=self.w_post, gate=self.gate, block_scale=0.5)
        dx, dh, du, a = block.ffn_backward_data(after["dy"], h, u, *self.weights, offsets=offsets)
        for g in self.grads:
            g.zero_()
        block.ffn_backward_weights(x, a, after["dy"], dh, du, self.n_experts, offsets, out=self.grads)
        before = block.norm_join_backward(after["dres"], dx, None, tokens, w_pre=self.w_pre)
        return before["dres"], {"w_pre": before["dw_pre"], "w_post": after["dw_post"], "gate": after["dgate"]}

    def step(self, small, lr: float):
        """AdamW on the shard from the row-major gradients, new codes and scales; a plain step on
        the small float32 parameters."""
        self.shard.step(self.hp, self.grads, self.codes, self.scales, fold_on_read=True)
        for name, g in small.items():
            getattr(self, name).sub_(g, alpha=lr)


def main(argv=None) -> list:
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=40)
    ap.add_argument("--experts", type=int, default=4)
    ap.add_argument("--width", type=int, default=512)
    ap.add_argument("--inner", type=int, default=256)
    ap.add_argument("--tokens", type=int, default=1024)
    ap.add_argument("--lr", type=float, default=5e-3)
    args = ap.parse_args(argv)

    import torch

    import blockwise_fp8_zero_fold_amd as fz

    hp = fz.Hparams(args.lr, 0.9, 0.95, 1e-8, 0.0, 1.0, 0, 1.0, 2.0, 0.5, 1000, 0, 0, 0.0, None)
    make = lambda seed: Layer(args.experts, args.width, args.inner, hp, seed)  # noqa: E731
    teacher, student = make(1), make(2)
    g = torch.Generator(device="cuda").manual_seed(3)
    tokens = torch.randn(args.tokens, args.width, device="cuda", generator=g).bfloat16()
    # tokens of each expert, already sorted: uneven loads
    cuts = torch.randint(0, args.tokens + 1, (args.experts - 1,), device="cuda", generator=g).sort().values
    offsets = torch.zeros(args.experts + 1, dtype=torch.int32, device="cuda")
    offsets[1:-1] = cuts
    offsets[-1] = args.tokens
    target, _ = teacher.forward(tokens, offsets)
    losses = []
    for step in range(args.steps):
        z, kept = student.forward(tokens, offsets)
        diff = z.float() - target.float()
        losses.append(float(diff.square().mean()))
        dz = (diff * (2.0 / args.tokens)).bfloat16()
        _, small = student.backward(dz, tokens, offsets, kept)
        student.step(small, 1e-3)
        if step % 10 == 0 or step + 1 == args.steps:
            print(f"step {step:4d}  loss {losses[-1]:.5f}", flush=True)
    return losses


if __name__ == "__main__":
    main()

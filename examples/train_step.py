"""A data-parallel training step from the products to the weights, on one GPU.

W replicas (rows of one gradient array) run a residual block

    z = x W1^T + b1,   h = gelu(z),   y = h W2^T + x

on their own tokens; their weight gradients land in the rows that the ZeRO-1
flush reads; the flush reduces each to the rank that owns it; and each owner
orthogonalises its whole gradient matrices (zc.Muon) and updates the weights.
Run it on a GPU:

    python examples/train_step.py            # a few steps, printing the loss
"""
from __future__ import annotations

import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import zero_collectives_gb300 as zc  # noqa: E402


class Block:
    """Weights of the block, W replicas' gradient rows, and the owners' optimizers."""

    def __init__(self, world: int = 4, width: int = 256, inner: int = 512, seed: int = 0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.world, self.width, self.inner = world, width, inner
        self.w1 = (torch.randn(inner, width, device="cuda", generator=g) / width ** 0.5).bfloat16()
        self.w2 = (torch.randn(width, inner, device="cuda", generator=g) / inner ** 0.5).bfloat16()
        self.b1 = torch.zeros(inner, device="cuda")
        # model order w1, b1, w2; gradients arrive in reverse (backward) order, in one bucket
        self.shapes = [(inner, width), (inner,), (width, inner)]
        self.numel = np.array([int(np.prod(s)) for s in self.shapes], np.int64)
        arrival, self.row_offset, pos = [2, 0, 1], np.zeros(3, np.int64), 0
        for p in arrival:
            self.row_offset[p] = pos
            pos += int(self.numel[p])
        tasks = np.zeros(3, zc.TASK_DTYPE)
        tasks["param_id"] = arrival
        tasks["offset"] = self.row_offset[arrival]
        tasks["numel"] = self.numel[arrival]
        self.rows = torch.zeros(world, pos, dtype=torch.bfloat16, device="cuda")
        self.ex = zc.Zero1Executor(world, self.numel, self.row_offset, [(0, tasks)], torch.bfloat16)
        # the rank that keeps each parameter (the first holder of one that straddles a partition boundary)
        self.keeper = [int(r) for r in self.ex.omap.holder_lo]
        self.muon = [zc.Muon([w for p, w in ((0, self.w1), (2, self.w2)) if self.keeper[p] == r]) for r in range(world)]

    def gradient(self, replica: int, param: int) -> torch.Tensor:
        """That replica's gradient of a parameter: a view of its row."""
        o = int(self.row_offset[param])
        return self.rows[replica, o:o + int(self.numel[param])].view(self.shapes[param])

    def replica_step(self, replica: int, x: torch.Tensor, target: torch.Tensor) -> torch.Tensor:
        """Forward and backward of one replica's tokens; returns the loss."""
        z = torch.empty(x.shape[0], self.inner, dtype=torch.bfloat16, device="cuda")
        h = zc.linear(x, self.w1, bias=self.b1, act="gelu", preact=z)
        y = zc.linear(h, self.w2, residual=x)
        err = y.float() - target.float()
        dy = (err * (2.0 / err.numel())).bfloat16()
        zc.linear_wgrad(dy, h, self.gradient(replica, 2))
        dz = zc.linear_dgrad(dy, self.w2, preact=z, act="gelu")
        db = torch.empty(self.inner, device="cuda")
        zc.linear_wgrad(dz, x, self.gradient(replica, 0), bias_grad=db)
        self.gradient(replica, 1).copy_(db)
        return err.square().mean()

    def step(self, xs, targets, lr: float = 0.02) -> torch.Tensor:
        """One optimizer step over every replica's tokens; returns the mean loss."""
        loss = torch.stack([self.replica_step(r, x, t) for r, (x, t) in enumerate(zip(xs, targets))]).mean()
        self.ex.flush_all(self.rows)  # mean over replicas, to the owners
        for rank in range(self.world):
            grads = [self.ex.grad.view(rank, p).view(self.shapes[p]) for p in (0, 2) if self.keeper[p] == rank]
            if grads:
                self.muon[rank].step(grads, lr)
            if self.keeper[1] == rank:
                self.b1.add_(self.ex.grad.view(rank, 1).float(), alpha=-lr)
        return loss


def main() -> None:
    block = Block()
    g = torch.Generator(device="cuda").manual_seed(1)
    shift = torch.randn(block.width, block.width, device="cuda", generator=g) / block.width ** 0.5
    xs = [torch.randn(384, block.width, device="cuda", generator=g).bfloat16() for _ in range(block.world)]
    targets = [(x.float() + torch.tanh(x.float() @ shift)).bfloat16() for x in xs]
    print(block.ex.omap.report())
    for step in range(20):
        loss = block.step(xs, targets)
        if step % 5 == 0 or step == 19:
            print(f"step {step:2d}  loss {float(loss):.4f}")


if __name__ == "__main__":
    main()

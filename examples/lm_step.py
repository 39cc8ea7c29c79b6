"""A data-parallel training step from token ids to the weights, on one GPU.

W replicas (rows of one gradient array) run a residual network over their own
tokens: an embedding, then blocks with norms on either side,

    h = N(x, pre),   y = gelu(h W1^T) W2^T,   x = s x + gate N(y, post),

and a last norm whose output is compared with given features.  Every gradient
lands in the rows that the ZeRO-1 flush reads, the embedding's included; the
flush reduces each parameter to the rank that owns it; the reduced gradients are
clipped together; and each owner updates what it owns, whole matrices of the
blocks by orthogonalised updates (zc.Muon), the rest by plain steps.  Run it on a
GPU:

    python examples/lm_step.py            # a few steps, printing the loss and the gradient norm
"""
from __future__ import annotations

import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import zero_collectives_gb300 as zc  # noqa: E402


class Model:
    """Weights, W replicas' gradient rows, and the owners' optimizers."""

    def __init__(self, world: int = 4, vocab: int = 1000, width: int = 128, inner: int = 256, blocks: int = 2, seed: int = 0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def matrix(rows, cols, scale):
            return (torch.randn(rows, cols, device="cuda", generator=g) * scale).bfloat16()

        self.world, self.blocks, self.scale, self.residual = world, blocks, width ** 0.5, 0.9
        self.params = {"embed": matrix(vocab, width, 1 / width ** 0.5), "norm0": torch.ones(width, device="cuda")}
        for i in range(blocks):
            self.params.update({f"w1.{i}": matrix(inner, width, 1 / width ** 0.5), f"w2.{i}": matrix(width, inner, 1 / inner ** 0.5),
                                f"post.{i}": torch.ones(width, device="cuda"), f"gate.{i}": torch.full((width,), 0.5, device="cuda"),
                                f"norm{i + 1}": torch.ones(width, device="cuda")})
        self.names = list(self.params)
        # gradients arrive in reverse (backward) order, in one bucket
        numel = np.array([self.params[n].numel() for n in self.names], np.int64)
        arrival, offset, pos = list(range(len(self.names)))[::-1], np.zeros(len(self.names), np.int64), 0
        for p in arrival:
            offset[p] = pos
            pos += int(numel[p])
        tasks = np.zeros(len(arrival), zc.TASK_DTYPE)
        tasks["param_id"], tasks["offset"], tasks["numel"] = arrival, offset[arrival], numel[arrival]
        self.rows = torch.zeros(world, pos, dtype=torch.bfloat16, device="cuda")
        self.at = {n: (int(o), int(o + k)) for n, o, k in zip(self.names, offset, numel)}
        self.ex = zc.Zero1Executor(world, numel, offset, [(0, tasks)], torch.bfloat16)
        self.clip = self.ex.grad_clip()
        # the rank that keeps each parameter (the first holder of one that straddles a partition boundary)
        self.keeper = {n: int(r) for n, r in zip(self.names, self.ex.omap.holder_lo)}
        self.matrices = [n for n in self.names if n.startswith("w")]
        self.muon = [zc.Muon([self.params[n] for n in self.matrices if self.keeper[n] == r]) for r in range(world)]

    def gradient(self, replica: int, name: str) -> torch.Tensor:
        """That replica's gradient of a parameter: a view of its row."""
        lo, hi = self.at[name]
        return self.rows[replica, lo:hi].view(self.params[name].shape)

    def replica_step(self, replica: int, ids: torch.Tensor, target: torch.Tensor, padding: int | None = None) -> torch.Tensor:
        """Forward and backward of one replica's tokens; returns the loss."""
        p, kept = self.params, []
        x = zc.embedding(ids, p["embed"], scale=self.scale)
        x, h = zc.block_norm(x, pre=p["norm0"])
        bottom = x
        for i in range(self.blocks):
            z = torch.empty(ids.numel(), p[f"w1.{i}"].shape[0], dtype=torch.bfloat16, device="cuda")
            a = zc.linear(h, p[f"w1.{i}"], act="gelu", preact=z)
            y = zc.linear(a, p[f"w2.{i}"])
            below = h
            x, h = zc.block_norm(x, y=y, post=p[f"post.{i}"], gate=p[f"gate.{i}"], residual_scale=self.residual, pre=p[f"norm{i + 1}"])
            kept.append((below, z, a, y, x))
        err = h.float() - target.float()
        dh, dx = (err * (2.0 / err.numel())).bfloat16(), None
        for i in reversed(range(self.blocks)):
            below, z, a, y, x = kept[i]
            dx, dy = zc.block_norm_grad(x, dr=dx, dh=dh, y=y, post=p[f"post.{i}"], gate=p[f"gate.{i}"], residual_scale=self.residual,
                                        pre=p[f"norm{i + 1}"], post_grad=self.gradient(replica, f"post.{i}"),
                                        gate_grad=self.gradient(replica, f"gate.{i}"), pre_grad=self.gradient(replica, f"norm{i + 1}"))
            zc.linear_wgrad(dy, a, self.gradient(replica, f"w2.{i}"))
            dz = zc.linear_dgrad(dy, p[f"w2.{i}"], preact=z, act="gelu")
            zc.linear_wgrad(dz, below, self.gradient(replica, f"w1.{i}"))
            dh = zc.linear_dgrad(dz, p[f"w1.{i}"])
        dx, _ = zc.block_norm_grad(bottom, dr=dx, dh=dh, pre=p["norm0"], pre_grad=self.gradient(replica, "norm0"))
        zc.embedding_grad(ids, dx, self.gradient(replica, "embed"), scale=self.scale, padding=padding)
        return err.square().mean()

    def step(self, ids, targets, lr: float = 0.02, max_norm: float = 1.0):
        """One optimizer step over every replica's tokens; returns the mean loss and
        the gradient norm with the factor of the clipping."""
        loss = torch.stack([self.replica_step(r, i, t) for r, (i, t) in enumerate(zip(ids, targets))]).mean()
        self.ex.flush_all(self.rows)  # mean over replicas, to the owners
        norm = self.clip.clip(max_norm)
        for rank in range(self.world):
            def reduced(name):
                return self.ex.grad.view(rank, self.names.index(name)).view(self.params[name].shape)
            grads = [reduced(n) for n in self.matrices if self.keeper[n] == rank]
            if grads:
                self.muon[rank].step(grads, lr)
            for n in self.names:
                if n not in self.matrices and self.keeper[n] == rank:
                    self.params[n].sub_(reduced(n), alpha=lr)
        return loss, norm


def main() -> None:
    model = Model()
    g = torch.Generator(device="cuda").manual_seed(1)
    features = torch.randn(1000, 128, device="cuda", generator=g)
    ids = [torch.randint(0, 1000, (384,), device="cuda", generator=g) for _ in range(model.world)]
    print(model.ex.omap.report())
    for step in range(20):
        loss, norm = model.step(ids, [features[i] for i in ids])
        if step % 5 == 0 or step == 19:
            print(f"step {step:2d}  loss {float(loss):.4f}  gradient norm {float(norm[0]):.4f} (scaled by {float(norm[1]):.3f})")


if __name__ == "__main__":
    main()

"""A bucket flush with the overlap promise after a product or an update.

The promise is about the call just before the flush; whatever ran before that
call is done once that call is.  So a flush that shares nothing with the call
before it may rely on the gradients that an earlier weight gradient wrote,
although it starts without waiting for the call before."""
import numpy as np
import pytest
import torch

import zero_collectives_gb300 as zc

pytestmark = pytest.mark.gpu
WORLD, M, N, K = 2, 16384, 4096, 1024  # a weight gradient of about 80 us


def randn(*shape, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, device="cuda", generator=g) * scale).bfloat16()


class Buckets:
    """Two buckets: a small one, and one that holds one [N, K] gradient."""

    def __init__(self):
        self.numel = np.array([4096, N * K], np.int64)
        self.start = np.array([0, 4096], np.int64)
        self.rows = torch.zeros(WORLD, int(self.numel.sum()), dtype=torch.bfloat16, device="cuda")
        self.rows[:, :4096] = randn(WORLD, 4096, seed=1)
        self.om = zc.build_owner_map(WORLD, [(None, self.numel)], True)
        self.grad = zc.GradBuffers(WORLD, self.om, self.numel, self.start, torch.bfloat16, fill=0.0)
        self.tasks = []
        for p in range(2):
            t = np.zeros(1, zc.TASK_DTYPE)
            t["param_id"], t["offset"], t["numel"] = p, 0, self.numel[p]
            self.tasks.append(t)
        self.dy, self.x = randn(M, N, seed=2, scale=1e-2), randn(M, K, seed=3)

    def flush(self, b, overlap):
        s = int(self.start[b])
        zc.flush_bucket(self.rows[:, s:s + int(self.numel[b])], self.tasks[b], self.om.owner,
                        self.grad.dst_table(self.tasks[b]), overlap=overlap)

    def wgrad(self):
        """Every replica's gradient, one after another (the second replica sees other tokens)."""
        for r in range(WORLD):
            zc.linear_wgrad(self.dy[r * 256:], self.x[r * 256:], self.rows[r, 4096:].view(N, K))

    def run(self, between, overlap):
        self.rows[:, 4096:] = 0
        for b in self.grad.buf:
            b.zero_()
        torch.cuda.synchronize()
        self.wgrad()
        between(overlap)
        self.flush(1, overlap)
        torch.cuda.synchronize()
        return [b.clone() for b in self.grad.buf]


@pytest.fixture(scope="module")
def buckets():
    return Buckets()


def calls():
    x, w = randn(1024, 2048, seed=4), randn(2048, 1024, seed=5, scale=0.03)
    wt, big = w.T.contiguous(), randn(4096, 1024, seed=12)
    token, odd = randn(1, 1024, seed=6), randn(100, 2049, seed=7)
    dy, dw, db = randn(300, 1000, seed=8), torch.zeros(1000, 2048, device="cuda"), torch.zeros(1000, device="cuda")
    g = {s: randn(*s, seed=9) for s in ((64, 200), (300, 400), (8, 1024, 1024))}
    weights = [randn(300, 400, seed=10), randn(64, 96, seed=11)]
    opt, grads = zc.Muon(weights), [randn(*v.shape, seed=13) for v in weights]
    return {
        "dgrad": lambda: zc.linear_dgrad(x, w, out=torch.empty(1024, 1024, dtype=torch.bfloat16, device="cuda")),
        "linear of one token": lambda: zc.linear(token, w),
        "linear of packed rows": lambda: zc.linear(odd[:, 1:], wt),
        "large linear": lambda: zc.linear(big, w),
        "wgrad with bias": lambda: zc.linear_wgrad(dy, x[:300], dw, bias_grad=db),
        "small newton_schulz": lambda: zc.newton_schulz(g[64, 200]),
        "newton_schulz one by one": lambda: zc.newton_schulz(g[300, 400]),
        "chained newton_schulz": lambda: zc.newton_schulz(g[8, 1024, 1024]),
        "muon": lambda: opt.step(grads, 0.01),
    }


@pytest.mark.parametrize("name", ["dgrad", "linear of one token", "linear of packed rows", "large linear", "wgrad with bias",
                                  "small newton_schulz", "newton_schulz one by one", "chained newton_schulz", "muon"])
def test_flush_overlapping_the_call_after_the_weight_gradient(buckets, name):
    call = calls()[name]
    call()
    want = buckets.run(lambda overlap: call(), False)
    assert all(bool(b.any()) for b in want[:1])
    for _ in range(3):
        got = buckets.run(lambda overlap: call(), True)
        assert all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip(got, want))
    assert zc.device_status() == 0


def test_flush_after_an_overlapping_flush_after_the_weight_gradient(buckets):
    """weight gradient of bucket 1, flush of bucket 0, flush of bucket 1: the first flush shares nothing with the
    weight gradient, the second nothing with the first."""
    def between(overlap):
        buckets.flush(0, overlap)

    want = buckets.run(between, False)
    for _ in range(3):
        got = buckets.run(between, True)
        assert all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip(got, want))
    assert zc.device_status() == 0

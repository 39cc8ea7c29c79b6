"""Clipping with no counted gradient: the norm is 0, the factor 1, and nothing is
scaled, whatever the threshold."""
import pytest
import torch

import zero_collectives_gb300 as zc

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [5, 3_000_000])  # one cluster's launch, and two launches
@pytest.mark.parametrize("max_norm", [0.0, 1e-9, 1.0])
@pytest.mark.parametrize("eps", [0.0, 1e-6])
@pytest.mark.parametrize("empty", [False, True])
def test_copies_alone_stay(n, max_norm, eps, empty):
    copy = torch.arange(1, n + 1, device="cuda", dtype=torch.float32)
    keep = copy.clone()
    counted = [copy[:0]] if empty else []
    assert zc.clip_grads(counted, max_norm, copies=[copy], eps=eps).tolist() == [0.0, 1.0]
    assert torch.equal(copy, keep)
    assert zc.GradClip(counted, [copy], eps=eps).clip(max_norm).tolist() == [0.0, 1.0] and torch.equal(copy, keep)


@pytest.mark.parametrize("n", [5, 3_000_000])
def test_counted_zeros_follow_the_formula(n):
    """A norm of 0 that was counted: c = min(1, max_norm / eps)."""
    z, copy = torch.zeros(n, device="cuda"), torch.ones(7, device="cuda")
    assert zc.clip_grads([z], 2.0 ** -21, copies=[copy], eps=2.0 ** -20).tolist() == [0.0, 0.5] and copy.tolist() == [0.5] * 7
    assert zc.clip_grads([z], 1.0, copies=[copy]).tolist() == [0.0, 1.0] and copy.tolist() == [0.5] * 7
    assert zc.clip_grads([z], 0.0, copies=[copy], eps=0.0).tolist() == [0.0, 1.0] and copy.tolist() == [0.5] * 7

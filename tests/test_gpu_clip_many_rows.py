"""Clipping of a matrix with as many narrow rows as there may be."""
import math

import pytest
import torch

import zero_collectives_gb300 as zc

pytestmark = pytest.mark.gpu
NORM = 7 * 2.0 ** -24  # as in test_gpu_clip.py


def test_the_most_rows():
    """One column of 2^31 - 1 rows (8.6 GB with the column beside it, which stays),
    before and behind another gradient."""
    rows = 2 ** 31 - 1
    wide = torch.empty(rows, 2, dtype=torch.bfloat16, device="cuda")
    g, beside = wide[:, :1], wide[:, 1]
    other = torch.full((3, 5), 1000.0, device="cuda")
    for grads in ([g, other], [other, g]):
        wide.fill_(0.5)
        other.fill_(1000.0)
        want = math.sqrt(0.25 * rows + 15e6)
        assert abs(float(zc.grad_norm(grads)) - want) <= NORM * want
        norm, c = zc.clip_grads(grads, 0.5 * want, eps=0.0).tolist()
        assert abs(norm - want) <= NORM * want and abs(c - 0.5) <= (NORM + 2.0 ** -24) * 0.5
        scaled = torch.full((1,), 0.5 * c, device="cuda").bfloat16()
        assert bool((g == scaled).all()) and bool((beside == 0.5).all())
        assert torch.equal(other, torch.full_like(other, 1000.0) * c)

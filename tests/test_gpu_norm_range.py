"""The block norms at the ends of the range that they take: elements of y and r up
to 3e18 whatever the width, and without eps rows whose mean square is 1e-34.

Tolerances are those of test_gpu_block_norm.py.  Gradients of large rows pass below
the smallest normal value (2^-126; dy is g / |r| / |y|), where a rounding is off by
up to half the smallest subnormal whatever the value: 2^-134 of bf16 for the stored
one, and 2^-150 of fp32 for each of the at most four products before it."""
import pytest
import torch

import zero_collectives_gb300 as zc
from tests import test_gpu_block_norm
from tests.test_gpu_block_norm import Case

pytestmark = pytest.mark.gpu
TINY = {torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -150}

# few rows, and rows through the rings; of known and any alignment, and the widest
SIZES = [(3, 128), (5, 777), (3, 1024), (2, 8192), (2, 16384), (6000, 777), (6000, 1024), (700, 4096), (420, 8191), (420, 16384), (420, 16383)]


@pytest.fixture(autouse=True)
def subnormal_outputs(monkeypatch):
    near = test_gpu_block_norm.near
    monkeypatch.setattr(test_gpu_block_norm, "near", lambda got, want, tol: near(got, want, tol + TINY[got.dtype] + 4 * 2.0 ** -150))


def both(c):
    c.check_forward(*c.forward())
    if c.dr is not None:
        c.dr.mul_(0.0)  # so that the norm's own part shows
    grads = c.grads()
    c.check_backward(*c.backward(grads), grads)
    assert zc.device_status() == 0


@pytest.mark.parametrize("m,d", SIZES)
@pytest.mark.parametrize("stream", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("value", [1e17, 1e18, 3e18])
@pytest.mark.parametrize("form", [dict(), dict(y=False), dict(gate=0, dr=False)], ids=str)
def test_large_rows(m, d, stream, value, form):
    """Rows of which every element is as large, beside ordinary ones, and no others."""
    c = Case(m, d, stream=stream, **form)
    for rows in (slice(None, None, 2), slice(1, None, 2)):
        for t in (c.x, c.y):
            if t is not None:
                t[rows] = t[rows].sign() * value
        both(c)


@pytest.mark.parametrize("m,d", SIZES)
def test_single_large_elements(m, d):
    """The squares of one element, and those of elements that one thread has."""
    c = Case(m, d, stream=torch.float32)
    c.x[0, d // 2] = 3e18
    c.y[m - 1, 7] = -3e18
    c.x[m // 2, :8] = 3e18
    both(c)


@pytest.mark.parametrize("m,d", SIZES)
@pytest.mark.parametrize("value", [1e-12, 1e-17])
def test_small_rows_without_eps(m, d, value):
    c = Case(m, d, stream=torch.float32, eps=0.0)
    for t in (c.x, c.y):
        t[::2] *= value
    both(c)

"""fp32 results of long reductions keep fp32 accuracy on either kernel.

Tolerance (2-norm, relative), for sums of random terms: an accumulator takes at
most 512 elements, 32 steps of 16, and each step drops at most a unit in the
last place of the partial sum, half of one on average (2^-24 of a partial sum at the
lower end of its binade); a run's partial sums average 2/3 of its end value, so
a run is off by at most 32 * 2^-24 * 2/3 = 1.3e-6 of itself.  The runs' errors
add as the runs do.  Up to 2048 runs are then added in fp32, each
addition off by 2^-25 of its sum on average, in quadrature: sqrt(2048) * 2^-25
* 2/3 < 0.9e-6 for the longest, 3e-7 up to 200 runs.  Together 2.2e-6."""
import math

import pytest
import torch

import zero_collectives_gb300 as zc

pytestmark = pytest.mark.gpu
TOL = 2.2e-6


def randn(*shape, seed, scale=1.0, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, device="cuda", generator=g) * scale).to(dtype)


def rel(got, want):
    return float((got.double() - want).norm() / want.norm())


@pytest.mark.parametrize("m,n,k", [(98304, 512, 256), (65536, 1024, 512), (1 << 20, 256, 256), (98304, 128, 128), (30000, 200, 72),
                                   (16384, 2048, 1024), (98304, 1024, 2048), (100001, 328, 264)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_wgrad(m, n, k, accumulate):
    dy, x = randn(m, n, seed=1, scale=1e-2), randn(m, k, seed=2)
    dw, db = randn(n, k, seed=3, dtype=torch.float32), randn(n, seed=4, dtype=torch.float32)
    want, want_db = dw.double() * accumulate, db.double() * accumulate
    for i in range(0, m, 1 << 18):
        part = dy[i:i + (1 << 18)].double()
        want, want_db = want + part.T @ x[i:i + (1 << 18)].double(), want_db + part.sum(0)
    other = dw.clone()
    zc.linear_wgrad(dy, x, dw, bias_grad=db, accumulate=accumulate)
    zc.linear_wgrad(dy, x, other, accumulate=accumulate)
    assert rel(dw, want) <= TOL and rel(other, want) <= TOL and rel(db, want_db) <= TOL
    assert zc.device_status() == 0


@pytest.mark.parametrize("m", [1, 9, 64, 200])
@pytest.mark.parametrize("n,k", [(98304, 1024), (200000, 136), (16392, 64)])
def test_dgrad_and_linear(m, n, k):
    """The gradient of a projection over a whole vocabulary, and a product that long."""
    dy, w = randn(m, n, seed=1), randn(n, k, seed=2, scale=1 / math.sqrt(n))
    want = dy.double() @ w.double()
    assert rel(zc.linear_dgrad(dy, w, out_dtype=torch.float32), want) <= TOL
    assert rel(zc.linear(dy, w.T.contiguous(), out_dtype=torch.float32), want) <= TOL
    z = randn(m, k, seed=3)
    relu = zc.linear_dgrad(dy, w, preact=z, act="relu", out_dtype=torch.float32)
    assert rel(relu, want * (z.double() > 0)) <= TOL
    assert zc.device_status() == 0

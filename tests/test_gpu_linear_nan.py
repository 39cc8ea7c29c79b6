"""A NaN reaches the results that depend on it, whatever the activation and the kernel, and no other."""
import pytest
import torch

import zero_collectives_gb300 as zc

pytestmark = pytest.mark.gpu
ACTS = ("none", "relu", "gelu", "silu")
# a few tokens (features on the lanes), the split kernel, the tile kernel with and without 16-byte aligned rows
SHAPES = [(6, 72, 100), (70, 72, 100), (4096, 2048, 128), (4096, 2047, 128)]


def randn(*shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, device="cuda", generator=g).bfloat16()


@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
def test_linear(m, n, k, act, out_dtype):
    x, w, r = randn(m, k, seed=1), randn(n, k, seed=2), randn(m, n, seed=3)
    for options in (dict(), dict(residual=r, preact=torch.empty(m, n, dtype=torch.bfloat16, device="cuda"))):
        clean = zc.linear(x, w, act=act, out_dtype=out_dtype, **options)
        bad = x.clone()
        bad[3, k - 1] = float("nan")
        y = zc.linear(bad, w, act=act, out_dtype=out_dtype, **options)
        assert bool(y[3].isnan().all())
        others = torch.arange(m, device="cuda") != 3
        assert torch.equal(y[others], clean[others])
        if options:
            assert bool(options["preact"][3].isnan().all())


@pytest.mark.parametrize("act", ["relu", "gelu", "silu"])
def test_bias(act):
    """From the bias: its own column."""
    for m, n, k in SHAPES:
        x, w, b = randn(m, k, seed=1), randn(n, k, seed=2), torch.zeros(n, device="cuda")
        b[5] = float("nan")
        y = zc.linear(x, w, bias=b, act=act)
        assert bool(y[:, 5].isnan().all()) and int(y.isnan().sum()) == m


@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("act", ["relu", "gelu", "silu"])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
def test_dgrad(m, n, k, act, out_dtype):
    """A NaN in the stored pre-activation gives a NaN in its own place; one in dy its own row, masked or not."""
    dy, w, z, r = randn(m, k, seed=1), randn(k, n, seed=2), randn(m, n, seed=3), randn(m, n, seed=4)
    for options in (dict(), dict(residual=r)):
        clean = zc.linear_dgrad(dy, w, preact=z, act=act, out_dtype=out_dtype, **options)
        bad = z.clone()
        bad[2, n - 1], bad[4, 0] = float("nan"), float("nan")
        dx = zc.linear_dgrad(dy, w, preact=bad, act=act, out_dtype=out_dtype, **options)
        assert bool(dx[2, n - 1].isnan()) and bool(dx[4, 0].isnan()) and int(dx.isnan().sum()) == 2
        assert bool(((dx == clean) | bad.isnan()).all())
        bad = dy.clone()
        bad[1, k - 1] = float("nan")
        dx = zc.linear_dgrad(bad, w, preact=z, act=act, out_dtype=out_dtype, **options)
        assert bool(dx[1].isnan().all()) and int(dx.isnan().sum()) == n


def test_signed_zeros_and_relu():
    """relu of -0 is +0; its gradient is 0 at both zeros."""
    z = torch.tensor([[-0.0, 0.0, 1.0, -1.0, float("inf"), -float("inf"), 1e-38, -1e-38]], device="cuda").bfloat16()
    eye, dy = torch.eye(8, dtype=torch.bfloat16, device="cuda"), torch.ones(1, 8, dtype=torch.bfloat16, device="cuda")
    assert torch.equal(zc.linear_dgrad(dy, eye, preact=z, act="relu").cpu(), torch.tensor([[0, 0, 1, 0, 1, 0, 1, 0]]).bfloat16())
    y = zc.linear(z[:, :4], eye[:4, :4], act="relu")
    assert torch.equal(y.cpu(), torch.tensor([[0, 0, 1, 0]]).bfloat16()) and not bool(y.signbit().any())

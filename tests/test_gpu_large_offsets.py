"""Matrices of more than 2^31 elements (and 2^32 bytes): the last rows are where
they belong."""
import math

import pytest
import torch

import zero_collectives_gb300 as zc

pytestmark = pytest.mark.gpu
ROWS, D = 2_200_003, 1024  # 2.25e9 elements


@pytest.fixture(autouse=True)
def memory():
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    yield
    torch.cuda.empty_cache()


def test_embedding():
    w = torch.zeros(ROWS, D, dtype=torch.bfloat16, device="cuda")
    ids = torch.tensor([0, ROWS - 1, ROWS - 2, 2097152, 2097151, ROWS - 1], device="cuda")
    w[ids] = torch.randn(6, D, device="cuda").bfloat16()
    assert torch.equal(zc.embedding(ids, w), w[ids])
    dy = torch.randn(6, D, device="cuda").bfloat16()
    want = w[ids].float()
    zc.embedding_grad(ids, dy, w, accumulate=True)
    for i, k in enumerate((0, None, ROWS - 2, 2097152, 2097151)):
        if k is not None:
            assert torch.equal(w[k], (want[i] + dy[i].float()).bfloat16())
    want = want[1] + (dy[1].float() + dy[5].float())
    assert float((w[ROWS - 1].float() - want).abs().max()) <= 2.0 ** -8 * float(want.abs().max())
    zc.embedding_grad(ids, dy, w)
    assert torch.equal(w[2097151], dy[4]) and not bool(w[ROWS - 3].any()) and not bool(w[1].any())
    assert zc.device_status() == 0


def test_block_norm():
    x = torch.zeros(ROWS, D, dtype=torch.bfloat16, device="cuda")
    x[-300:], x[:10] = torch.randn(300, D, device="cuda"), torch.randn(10, D, device="cuda")
    pre = torch.rand(D, device="cuda")
    _, h = zc.block_norm(x, pre=pre)
    _, few = zc.block_norm(x[-300:], pre=pre)
    assert torch.equal(h[:10], zc.block_norm(x[:10], pre=pre)[1])
    # the two ways of covering a row add its squares in another order: one rounding apart
    assert float((h[-300:].float() - few.float()).abs().max()) <= 2.0 ** -7 * float(few.float().abs().max())
    assert not bool(h[5000:6000].any())
    g = torch.zeros(D, device="cuda")
    dx, _ = zc.block_norm_grad(x, dh=h, pre=pre, pre_grad=g, dx=h)
    part = torch.zeros(D, device="cuda")
    want, _ = zc.block_norm_grad(x[-300:], dh=few, pre=pre, pre_grad=part)
    assert float((dx[-300:].float() - want.float()).abs().max()) <= 2.0 ** -6 * float(want.float().abs().max())
    assert bool(torch.isfinite(g).all()) and bool((g > 0.9 * part).all())


def test_gradient_norm():
    g = torch.ones(ROWS * D, dtype=torch.bfloat16, device="cuda")
    want = math.sqrt(g.numel())
    assert abs(float(zc.grad_norm([g])) / want - 1) < 1e-6
    zc.clip_grads([g], want / 2, eps=0.0)
    assert bool((g[-4096:] == 0.5).all()) and bool((g[:4096] == 0.5).all()) and bool((g[2 ** 31 - 2048:2 ** 31 + 2048] == 0.5).all())
    wide = torch.ones(5, 2 ** 29, dtype=torch.bfloat16, device="cuda")[:, :1000]
    assert abs(float(zc.grad_norm([wide])) / math.sqrt(5000) - 1) < 1e-6

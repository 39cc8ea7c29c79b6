"""Bias gradients whose sums are exact in fp32 in any order: a value of dy read
from another stage of the pipeline, twice or not at all, changes the result.

dy holds integers of magnitude 0 to 64 that depend on the token and the
column; every partial sum stays below 2^24 and is exact, and so is the product with a
one-hot x."""
import pytest
import torch

import zero_collectives_gb300 as zc

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m,n,k", [(16384, 4096, 1024), (16383, 4096, 1000), (8192, 2048, 512), (20000, 1500, 2048), (4096, 8192, 256),
                                   (700, 8000, 2048), (64, 16384, 1024), (65, 2304, 4096), (400, 256, 65536)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_integers(m, n, k, dtype):
    i = torch.arange(m, device="cuda")[:, None]
    j = torch.arange(n, device="cuda")[None, :]
    # the block of 64 tokens decides the value together with the token's and the column's places
    dy = (((i // 64) * 37 + (i % 64) * 11 + j * 5) % 129 - 64).bfloat16()
    x = torch.zeros(m, k, dtype=torch.bfloat16, device="cuda")
    x[torch.arange(min(m, k), device="cuda"), torch.arange(min(m, k), device="cuda")] = 1
    want = dy.double().sum(0).float()
    want_dw = torch.zeros(n, k, device="cuda")
    want_dw[:, :min(m, k)] = dy[:min(m, k)].float().T
    for _ in range(4):
        dw, db = torch.full((n, k), float("nan"), dtype=dtype, device="cuda"), torch.full((n,), float("nan"), device="cuda")
        zc.linear_wgrad(dy, x, dw, bias_grad=db)
        assert torch.equal(db, want)
        assert torch.equal(dw.float(), want_dw)
    start = torch.arange(n, device="cuda").float()
    db = start.clone()
    zc.linear_wgrad(dy, x, dw, bias_grad=db, accumulate=True)
    assert torch.equal(db, start + want) and torch.equal(dw.float(), 2 * want_dw)
    assert zc.device_status() == 0

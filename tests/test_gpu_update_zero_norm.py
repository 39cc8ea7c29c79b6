"""Zero matrices with eps = 0: the update is zero, on every path (one launch for small matrices, a launch
per product, all products chained)."""
import pytest
import torch

import zero_collectives_gb300 as zc

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("batch,m,n", [(3, 48, 80), (2, 20, 1999), (2, 300, 400), (9, 1024, 1024), (3, 700, 130)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_newton_schulz(batch, m, n, dtype):
    g = torch.randn(batch, m, n, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).to(dtype)
    clean = zc.newton_schulz(g, eps=0.0)
    g[1] = 0
    got = zc.newton_schulz(g, eps=0.0)
    assert not bool(got[1].any())
    assert all(torch.equal(got[k], clean[k]) for k in range(batch) if k != 1)
    assert bool(got[0].isfinite().all()) and bool(got[0].any())
    g[1, 0, 0] = float("nan")
    assert bool(zc.newton_schulz(g, eps=0.0)[1].isnan().all())


def test_muon_step():
    shapes = [(64, 96), (300, 400), (300, 400)]
    w = [torch.full(s, 2.0, device="cuda") for s in shapes]
    m, g = [torch.zeros(s, device="cuda") for s in shapes], [torch.zeros(s, device="cuda") for s in shapes]
    zc.muon_step(w, m, g, lr=0.5, weight_decay=0.5, eps=0.0)
    assert all(bool((x == 1.5).all()) for x in w) and not any(bool(x.any()) for x in m)

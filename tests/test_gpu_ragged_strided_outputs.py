"""Outputs that are views of wider rows, or of one row among other data: whatever lies beside them keeps its
bits.  The widths end inside a group of 16 bytes, where a bulk copy would write the whole group."""
import math

import pytest
import torch

import zero_collectives_gb300 as zc

pytestmark = pytest.mark.gpu
BITS = {torch.bfloat16: torch.int16, torch.float32: torch.int32}


def randn(*shape, seed, scale=1.0, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, device="cuda", generator=g) * scale).to(dtype)


class Framed:
    """A [rows, cols] view with row stride ld, among -0, NaN, the smallest subnormal and 7."""

    def __init__(self, rows, cols, ld, dtype, content=None, lead=16):
        n = lead + rows * ld + 64
        pattern = torch.tensor([-0.0, float("nan"), 0.0, 7.0], device="cuda").to(dtype)
        self.flat = pattern.repeat(n // 4 + 1)[:n].clone()
        self.flat.view(BITS[dtype])[2::4] = 1
        self.view = self.flat.as_strided((rows, cols), (ld, 1), lead)
        if content is not None:
            self.view.copy_(content)
        self.inside = torch.zeros(n, dtype=torch.bool, device="cuda")
        self.inside.as_strided((rows, cols), (ld, 1), lead).fill_(True)
        self.before = self.flat.clone()

    def check(self, want, tol):
        assert float((self.view.double() - want).norm()) <= tol * float(want.norm())
        assert bool(((self.view.double() - want).abs() <= 8 * tol * (want.abs() + want.abs().mean())).all())
        a, b = (t.view(BITS[t.dtype])[~self.inside] for t in (self.flat, self.before))
        assert torch.equal(a, b), "data beside the output changed"


TOL = {torch.bfloat16: 2.0 ** -8, torch.float32: 1e-5}  # one rounding; an fp32 sum of up to 4096 terms with room
WIDTHS = [5, 7, 63, 65, 129, 515, 1025, 2049, 2050, 2051, 2052, 2053, 2055, 2111, 2113, 4093]


@pytest.mark.parametrize("n", WIDTHS)
@pytest.mark.parametrize("m", [3, 70, 333, 4096])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_linear(n, m, dtype):
    k = 64
    ld = (n + 15) // 16 * 16 + 16
    x, w, r, b = randn(m, k, seed=1), randn(n, k, seed=2, scale=1 / 8), randn(m, ld, seed=3)[:, :n], randn(n, seed=4)
    z64 = x.double() @ w.double().T
    y = Framed(m, n, ld, dtype)
    zc.linear(x, w, out=y.view)
    y.check(z64, TOL[dtype])
    y, z = Framed(m, n, ld, dtype), Framed(m, n, ld, torch.bfloat16)
    zc.linear(x, w, bias=b, act="silu", residual=r, preact=z.view, out=y.view)
    z.check(z64 + b.double(), TOL[torch.bfloat16])
    z64 = z64 + b.double()
    y.check(z64 * torch.sigmoid(z64) + r.double(), 2.0 ** -8)
    if dtype == torch.bfloat16:  # in place
        y = Framed(m, n, ld, dtype, r)
        zc.linear(x, w, residual=y.view, out=y.view)
        y.check(x.double() @ w.double().T + r.double(), TOL[dtype])
    assert zc.device_status() == 0


@pytest.mark.parametrize("k", WIDTHS)
@pytest.mark.parametrize("m", [3, 333, 4096])
def test_dgrad(k, m):
    n, ld = 128, (k + 15) // 16 * 16 + 16
    dy, w, z = randn(m, n, seed=1), randn(n, k, seed=2, scale=1 / math.sqrt(n)), randn(m, ld, seed=3)[:, :k]
    for dtype in (torch.bfloat16, torch.float32):
        dx = Framed(m, k, ld, dtype)
        zc.linear_dgrad(dy, w, preact=z, act="relu", out=dx.view)
        dx.check(dy.double() @ w.double() * (z.double() > 0), TOL[dtype])
    assert zc.device_status() == 0


@pytest.mark.parametrize("k", WIDTHS)
@pytest.mark.parametrize("m,n", [(19, 214), (64, 2000), (1000, 1), (4096, 1), (300, 1030)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("accumulate", [False, True])
def test_wgrad(k, m, n, dtype, accumulate):
    """Among them a single row at an aligned place of a gradient row, with the next parameter right behind it."""
    ld = (k + 15) // 16 * 16 + (16 if n > 1 else 0)
    dy, x = randn(m, n, seed=1), randn(m, k, seed=2)
    old = randn(n, k, seed=3, dtype=dtype) if accumulate else None
    want = dy.double().T @ x.double() + (old.double() if accumulate else 0)
    for with_bias in (False, True):
        dw, db = Framed(n, k, ld, dtype, old), Framed(1, n, n, torch.float32)
        zc.linear_wgrad(dy, x, dw.view, bias_grad=db.view[0] if with_bias else None, accumulate=accumulate and not with_bias)
        if with_bias:
            db.check(dy.double().sum(0)[None], 1e-5)
            dw.check(dy.double().T @ x.double(), TOL[dtype])
        else:
            dw.check(want, TOL[dtype])
    assert zc.device_status() == 0

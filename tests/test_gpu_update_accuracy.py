"""What the header says about the accuracy of orthogonalised updates: five steps are off by at most 2.8e-3 of
the result (tests/test_gpu_muon.py derives it; for short sides from 16 on) plus an absolute part that shows where |G|_F is far below eps.

The absolute part: X's entries are stored times a power of two s >= sqrt(c / 2) (c the long side) in terms no finer than
fp16's subnormal spacing, so each of the five stored X is off by at most 2^-25 / s an entry, sqrt(r c) 2^-25 / s <=
sqrt(2 r) 2^-25 in the norm; what follows multiplies it by 3.4445 a step at most, 3.4445^5 + ... + 3.4445 = 682 in
all: 682 * 2^-25 * sqrt(2 r) = 2.9e-5 sqrt(r), where an orthogonal matrix has the norm sqrt(r)."""
import math

import pytest
import torch

import zero_collectives_gb300 as zc
from tests.test_gpu_muon import TOL, ns64

pytestmark = pytest.mark.gpu
ABSOLUTE = 682 * 2.0 ** -25 * math.sqrt(2)


def randn(*shape, seed):
    return torch.randn(*shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed))


@pytest.mark.parametrize("shape", [(100, 300), (300, 400), (1024, 1024), (2500, 300), (12, 1024, 1024), (6, 512, 2048)])
def test_norms_from_far_below_eps_to_far_above(shape):
    g = randn(*shape, seed=1)
    g = g / g.flatten(-2).norm(dim=-1).max()
    r = min(shape[-2:])
    for k in (8, 2, 0, -1, -2, -3, -4, -5, -6, -9):
        x = g * (1e-7 * 10.0 ** k)
        want = ns64(x)
        off = (zc.newton_schulz(x, out=torch.empty_like(x)).double() - want).flatten(-2 if len(shape) == 3 else 0).norm(dim=-1)
        size = want.flatten(-2 if len(shape) == 3 else 0).norm(dim=-1)
        assert bool((off <= TOL * size + ABSOLUTE * math.sqrt(r)).all()), k


def test_a_matrix_alone_and_beside_others():
    """The other shapes of a call may decide how a matrix's products run: the result is as accurate, and the same
    call gives the same bits."""
    def step(shapes):
        ws, gs = [torch.zeros(s, device="cuda") for s in shapes], [randn(*s, seed=sum(s)) for s in shapes]
        zc.muon_step(ws, [torch.zeros(s, device="cuda") for s in shapes], gs, lr=1.0, scale=1.0)
        return ws, gs

    for others in ([], [(300, 500)], [(512, 512)] * 8, [(64, 100), (1000, 300), (900, 900), (2048, 300), (260, 1024)]):
        shapes = [(640, 768)] + others
        ws, gs = step(shapes)
        for w, g in zip(ws, gs):
            want = ns64(g)
            assert float((-w.double() - want).norm()) <= TOL * float(want.norm())
        assert all(torch.equal(a, b) for a, b in zip(ws, step(shapes)[0]))
    assert zc.device_status() == 0

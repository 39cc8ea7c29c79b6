"""Orthogonalised updates against the 64-bit iteration.

Tolerance (2-norm, relative): each of the five steps rounds the off-diagonal
parts of A and of the polynomial, and the X they multiply, to fp16 (unit
roundoff 2^-11, root mean square 2^-11 / sqrt(3) of an ulp-sized value); two
such roundings a step at full strength and no cancellation between steps give
5 * 2 * 2^-11 / sqrt(3) = 2.8e-3.  A bf16 result adds its own rounding,
2^-8 / sqrt(3) = 2.3e-3 at most."""
import math

import pytest
import torch

import zero_collectives_gb300 as zc

pytestmark = pytest.mark.gpu
TOL = 5 * 2 * 2.0 ** -11 / math.sqrt(3)
TOL_BF16 = TOL + 2.0 ** -8 / math.sqrt(3)
A, B, C = 3.4445, -4.7750, 2.0315


def ns64(g, steps=5, eps=1e-7, coeffs=(A, B, C)):
    a, b, c = coeffs
    x = g.double()
    tall = x.shape[-2] > x.shape[-1]
    x = x.mT if tall else x
    x = x / (x.square().sum((-2, -1), keepdim=True).sqrt() + eps)
    for _ in range(steps):
        gram = x @ x.mT
        x = a * x + (b * gram + c * gram @ gram) @ x
    return x.mT if tall else x


def gradient(*shape, seed, scale=1e-3, rank=4, dtype=torch.float32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.randn(*shape, device="cuda", generator=g)
    u = torch.randn(*shape[:-1], rank, device="cuda", generator=g)
    v = torch.randn(*shape[:-2], rank, shape[-1], device="cuda", generator=g)
    return ((t + u @ v) * scale).to(dtype)


def rel(got, want):
    return float((got.double() - want).norm() / want.norm())


SHAPES = [(1, 1), (1, 77), (50, 1), (2, 3), (8, 8), (63, 65), (64, 64), (127, 129), (128, 333), (333, 128), (256, 256),
          (300, 1000), (1000, 300), (512, 512), (1024, 256), (777, 1535), (2048, 130), (100, 2048), (2048, 128),
          (5, 1999), (128, 2049), (129, 140), (90, 513)]


@pytest.mark.parametrize("m,n", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_newton_schulz(m, n, dtype):
    g = gradient(m, n, seed=m + n, dtype=dtype)
    want = ns64(g)
    out = zc.newton_schulz(g, out=torch.empty(m, n, dtype=torch.float32, device="cuda"))
    assert rel(out, want) <= TOL
    assert rel(zc.newton_schulz(g), want) <= TOL_BF16
    assert zc.device_status() == 0


@pytest.mark.parametrize("scale", [1e-6, 1.0, 1e6, 1e15])
def test_newton_schulz_magnitudes(scale):
    g = gradient(96, 200, seed=1, scale=scale)
    assert rel(zc.newton_schulz(g), ns64(g)) <= TOL_BF16


@pytest.mark.parametrize("steps,coeffs", [(1, None), (3, None), (10, (2.0, -1.5, 0.5)), (2, (1.5, -0.5, 0.0))])
def test_newton_schulz_steps_and_coefficients(steps, coeffs):
    g = gradient(100, 140, seed=2)
    got = zc.newton_schulz(g, steps=steps, coeffs=coeffs, out=torch.empty_like(g))
    assert rel(got, ns64(g, steps, coeffs=coeffs or (A, B, C))) <= TOL * max(1.0, steps / 5)


def test_ill_conditioned():
    """A spectrum falling as 1/k over 256 directions, where plain 16-bit iterations lose 1e-2."""
    g = torch.Generator(device="cuda").manual_seed(3)
    u = torch.linalg.qr(torch.randn(256, 256, device="cuda", generator=g))[0]
    v = torch.linalg.qr(torch.randn(400, 256, device="cuda", generator=g))[0]
    m = (u / torch.arange(1, 257, device="cuda")) @ v.T
    assert rel(zc.newton_schulz(m, out=torch.empty_like(m)), ns64(m)) <= TOL


@pytest.mark.parametrize("batch", [1, 3, 70])
def test_batches(batch):
    g = gradient(batch, 40, 72, seed=4)
    want = ns64(g)
    got = zc.newton_schulz(g)
    for k in range(batch):
        assert rel(got[k], want[k]) <= TOL_BF16


def test_strides():
    wide = gradient(3, 60, 100, seed=5)
    g = wide[:, :, 7:84]
    holder = torch.full((3, 61, 81), 7.0, device="cuda")
    out = holder[:, :60, 2:79]
    zc.newton_schulz(g, out=out)
    for k in range(3):
        assert rel(out[k], ns64(g[k])) <= TOL
    holder[:, :60, 2:79] = 7.0
    assert bool((holder == 7.0).all()), "elements outside the view were written"


def test_zero_and_special_matrices():
    g = gradient(4, 48, 80, seed=6)
    clean = zc.newton_schulz(g)
    g[1] = 0
    g[2, 5, 7] = float("nan")
    got = zc.newton_schulz(g)
    assert not bool(got[1].any())
    assert bool(torch.isnan(got[2]).all())
    assert torch.equal(got[0], clean[0]) and torch.equal(got[3], clean[3])
    g[2, 5, 7] = float("inf")
    got = zc.newton_schulz(g)
    assert bool(torch.isnan(got[2]).all()) and torch.equal(got[0], clean[0])


def test_empty():
    assert zc.newton_schulz(torch.zeros(0, 5, device="cuda")).shape == (0, 5)
    assert zc.newton_schulz(torch.zeros(0, 4, 5, device="cuda")).shape == (0, 4, 5)
    zc.muon_step([], [], [], lr=0.1)


def muon64(w, m, g, lr, mu, nesterov, wd, scale):
    m1 = mu * m.double() + g.double()
    u = g.double() + mu * m1 if nesterov else m1
    return (1 - lr * wd) * w.double() - lr * scale * ns64(u), m1


@pytest.mark.parametrize("wdt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("gdt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("nesterov,wd,rule", [(True, 0.0, "spectral"), (False, 0.1, "rms"), (True, 0.1, 0.7)])
def test_muon_step(wdt, gdt, nesterov, wd, rule):
    shapes = [(64, 64), (100, 333), (333, 100), (64, 64), (1, 9), (0, 4), (257, 64), (64, 64)]
    ws = [gradient(*s, seed=10 + i, scale=0.02, rank=1).to(wdt) if s[0] else torch.zeros(s, dtype=wdt, device="cuda")
          for i, s in enumerate(shapes)]
    ms = [gradient(*s, seed=30 + i) if s[0] else torch.zeros(s, device="cuda") for i, s in enumerate(shapes)]
    gs = [gradient(*s, seed=50 + i).to(gdt) if s[0] else torch.zeros(s, dtype=gdt, device="cuda")
          for i, s in enumerate(shapes)]
    lr = 0.03
    want = [muon64(w, m, g, lr, 0.9, nesterov, wd, zc.update_scale(*s, rule)) if s[0] else None
            for w, m, g, s in zip(ws, ms, gs, shapes)]
    keep, m_old = [g.clone() for g in gs], [m.clone() for m in ms]
    zc.muon_step(ws, ms, gs, lr=lr, momentum=0.9, nesterov=nesterov, weight_decay=wd, scale=rule)
    for w, m, m0, e, s, g, g0 in zip(ws, ms, m_old, want, shapes, gs, keep):
        assert torch.equal(g, g0)
        if e is None:
            continue
        # momentum: two fp32 roundings, of the result and of mu times the old momentum
        assert bool(((m.double() - e[1]).abs() <= 2.0 ** -22 * (e[1].abs() + 0.9 * m0.double().abs())).all())
        last = 2.0 ** -8 if wdt == torch.bfloat16 else 2.0 ** -22
        update = lr * zc.update_scale(*s, rule) * math.sqrt(min(s)) * 1.3  # |X|_F, singular values below 1.3
        assert float((w.double() - e[0]).norm()) <= last * float(e[0].norm()) + TOL * update


def test_muon_weights_inside_a_larger_buffer():
    """Weights and gradients as views of flat buffers at odd offsets."""
    flat = torch.full((2, 5000), 3.0, device="cuda")
    w, g = flat[0, 3:3 + 40 * 70].view(40, 70), flat[1, 5:5 + 40 * 70].view(40, 70)
    w.copy_(gradient(40, 70, seed=1, scale=0.02))
    g.copy_(gradient(40, 70, seed=2))
    m = torch.zeros(40, 70, device="cuda")
    want = muon64(w, m, g, 0.1, 0.95, True, 0.0, 1.0)[0]
    zc.muon_step([w], [m], [g], lr=0.1)
    assert float((w.double() - want).norm()) <= 2.0 ** -22 * float(want.norm()) + TOL * 0.1 * math.sqrt(40) * 1.3
    assert bool((flat[0, :3] == 3).all()) and bool((flat[0, 2803:] == 3).all())


def test_muon_object_streams_and_graph():
    shapes = [(64, 96), (64, 96), (130, 50)]

    def fresh():
        return [gradient(*s, seed=i, scale=0.02).bfloat16() for i, s in enumerate(shapes)]

    gs = [gradient(*s, seed=9 + i).bfloat16() for i, s in enumerate(shapes)]
    a, b, c = (zc.Muon(fresh(), weight_decay=0.1) for _ in range(3))
    for _ in range(3):
        a.step(gs, lr=0.02)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        b.step(gs, lr=0.02, stream=s)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.step(gs, lr=0.02)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for x, y, z in zip(a.weights + a.momenta, b.weights + b.momenta, c.weights + c.momenta):
        assert torch.equal(x, y) and torch.equal(x, z)


@pytest.mark.parametrize("shapes", [[(1024, 1024)] * 8, [(700, 1300), (1300, 700), (700, 1300), (900, 900)] * 6,
                                    [(300, 4000)] * 3 + [(257, 2500)] * 5 + [(1030, 520)] * 4 + [(64, 96)] * 2,
                                    [(512 + 8 * i, 777) for i in range(11)], [(260, 1000)] * 70])
def test_many_large_matrices(shapes):
    """Batches whose products run chained in one launch: several shapes, ragged tiles, more shapes or matrices than a launch takes."""
    ws = [gradient(*s, seed=i, scale=0.02, rank=1) for i, s in enumerate(shapes)]
    gs = [gradient(*s, seed=100 + i).bfloat16() for i, s in enumerate(shapes)]
    ms = [torch.zeros(s, device="cuda") for s in shapes]
    w0 = [w.clone() for w in ws]
    zc.muon_step(ws, ms, gs, lr=0.1, scale=1.0)
    for w, w1, g, s in zip(w0, ws, gs, shapes):
        want = muon64(w, torch.zeros(s, device="cuda"), g, 0.1, 0.95, True, 0.0, 1.0)[0]
        assert float((w1.double() - want).norm()) <= 2.0 ** -22 * float(want.norm()) + TOL * 0.1 * math.sqrt(min(s)) * 1.3
    again = [w.clone() for w in w0]
    zc.muon_step(again, [torch.zeros(s, device="cuda") for s in shapes], gs, lr=0.1, scale=1.0)
    assert all(torch.equal(x, y) for x, y in zip(again, ws)), "two runs differ"
    assert zc.device_status() == 0


@pytest.mark.parametrize("shapes", [[(40, 4096)] * 48 + [(1500, 1500)] * 4, [(992, 1248)] * 10, [(130, 2080)] * 20 + [(2080, 600)] * 6])
def test_chained_tiles_of_short_reductions_and_ragged_rows(shapes):
    """Reductions of one to three blocks, whose tiles follow one another closely, and row tails beside whole 32-column chunks."""
    gs = [gradient(*s, seed=200 + i) for i, s in enumerate(shapes)]
    ws, ms = [torch.zeros_like(g) for g in gs], [torch.zeros_like(g) for g in gs]
    zc.muon_step(ws, ms, gs, lr=1.0, scale=1.0)
    for w, g in zip(ws, gs):
        assert rel(-w, ns64(g)) <= TOL
    assert zc.device_status() == 0

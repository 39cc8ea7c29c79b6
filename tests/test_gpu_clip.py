"""The global gradient norm and clipping against 64-bit ones.

Tolerances.  Sums of squares: a chunk adds at most 32 squares in four chains of
fused steps (8 + 2 roundings of 2^-24, all terms positive), chunks are added with
an error term (2^-23 in all), the rest in fp64; the root halves that, and the
result is rounded once: 7 * 2^-24.  Scaled values: the factor's own 7 * 2^-24 and
its rounding, one for the product in fp32, one to the type."""
import math

import numpy as np
import pytest
import torch

import zero_collectives_gb300 as zc
from datagen import workloads

pytestmark = pytest.mark.gpu
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -150}  # half the smallest value
NORM = 7 * 2.0 ** -24


def grad(rows, cols, seed, scale=1e-2, dtype=torch.bfloat16, pad=0, shift=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = (torch.randn(rows * (cols + pad) + shift, device="cuda", generator=g) * scale).to(dtype)
    return t[shift:].view(rows, cols + pad)[:, :cols]


def norm64(grads):
    return math.sqrt(sum(float(g.double().square().sum()) for g in grads))


def check(grads, copies=(), share=0.5, eps=1e-6):
    """Norm and clipping to a share of it."""
    want = norm64(grads)
    before = [g.double() for g in (*grads, *copies)]
    assert abs(float(zc.grad_norm(grads)) - want) <= NORM * want
    limit = share * want if want else 1.0
    got = zc.clip_grads(grads, limit, copies, eps=eps).tolist()
    limit = float(np.float32(limit))
    c = min(1.0, limit / (want + float(np.float32(eps)))) if want else 1.0
    assert abs(got[0] - want) <= NORM * want and abs(got[1] - c) <= (NORM + 2.0 ** -24) * c
    for g, b in zip((*grads, *copies), before):
        if share > 1:
            assert torch.equal(g.double(), b)
        tol = (HALF[g.dtype] + 10 * 2.0 ** -24) * (b * c).abs() + 2 * TINY[g.dtype]
        assert bool(((g.double() - b * c).abs() <= tol).all())


SETS = [
    [(1, 1)], [(1, 7)], [(1, 8192)], [(1, 8193)], [(3, 5), (1, 1), (100, 333)], [(2, 50000), (7, 1)], [(300, 1000), (64, 64), (1, 100003)],
    [(1, 31)] * 40, [(5, 77)] * 300, [(1, 1000)] * 800, [(4000, 3000)]]


@pytest.mark.parametrize("shapes", SETS, ids=lambda s: f"{len(s)}x{s[0][0]}x{s[0][1]}")
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("share", [0.5, 2.0])
def test_sets(shapes, dtype, share):
    check([grad(r, c, i, dtype=dtype) for i, (r, c) in enumerate(shapes)], share=share)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shift", [0, 1, 3, 8])
@pytest.mark.parametrize("rows,cols,pad", [(5, 3, 1), (700, 1, 3), (40, 255, 2), (40, 256, 8), (33, 1000, 5), (9, 20000, 7), (3, 70001, 9), (2, 8192, 8)])
def test_strided_rows(rows, cols, pad, shift, dtype):
    """What lies between the rows is neither counted nor scaled."""
    g = grad(rows, cols, 1, dtype=dtype, pad=pad, shift=shift)
    gap = g.as_strided((rows - 1, pad), (cols + pad, 1), g.storage_offset() + cols)
    gap.fill_(1e4)
    check([g, grad(7, 9, 2)])
    assert bool((gap == gap.flatten()[0]).all()) and float(gap.flatten()[0]) > 9e3


def test_mixed_types_and_copies():
    a, b, c = grad(30, 50, 1), grad(20, 999, 2, dtype=torch.float32), grad(1, 4000, 3)[0]
    check([a, b, c, torch.zeros(0, device="cuda")], copies=[a.clone(), b.clone()])
    wide = grad(40, 96, 4)
    check([wide[:, :30], wide[:, 30:64]], copies=[wide[:, 64:]])  # side by side in one matrix
    v = grad(1, 400, 5)[0][::2]  # a strided vector
    check([v])
    check([grad(4, 6 * 8, 6).view(4, 6, 8)])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_many_copies(dtype):
    """Copies in launches with and without counted gradients."""
    check([grad(300, 1000, 1, dtype=dtype)], copies=[grad(400, 5000, 2, dtype=dtype), grad(70, 33, 3, dtype=dtype, pad=5)])
    check([grad(1, 50 + i, i, dtype=dtype) for i in range(500)], copies=[grad(1, 50 + i, i, dtype=dtype) for i in range(1200)])
    check([grad(1, 9, 1)], copies=[grad(1, 10 + i, i, dtype=dtype) for i in range(800)])


@pytest.mark.parametrize("n", [5000, 3_000_000])
def test_the_whole_range_of_values(n):
    """Squares that overflow or underflow fp32, alone and beside ordinary ones."""
    for scale in (1e-38, 1e-30, 1e-22, 1e-12, 1e10, 1e18, 1e25, 1e34):
        for dtype in (torch.bfloat16, torch.float32):
            check([(torch.randn(n, device="cuda").clamp(-3, 3) * scale).to(dtype)], eps=0.0)
    big = torch.full((100000,), 1.5e18, device="cuda")
    assert abs(float(zc.grad_norm([big])) / (1.5e18 * 100000 ** 0.5) - 1) < 1e-6
    tiny = torch.full((33,), 1e-45, device="cuda")  # the smallest subnormal
    assert abs(float(zc.grad_norm([tiny.repeat(10000)])) / (float(tiny[0]) * 330000 ** 0.5) - 1) < 2.0 ** -9  # a subnormal norm has few bits
    check([grad(1, 3000, 1, scale=1e-25), grad(1, 3000, 2, scale=1e25), grad(1, 3000, 3)])


def test_nothing_to_clip():
    z = torch.zeros(5000, device="cuda")
    assert zc.clip_grads([z], 1.0).tolist() == [0.0, 1.0] and zc.clip_grads([z], 0.0, eps=0.0).tolist() == [0.0, 1.0]
    assert zc.clip_grads([], 1.0).tolist() == [0.0, 1.0] and float(zc.grad_norm([])) == 0.0
    assert float(zc.grad_norm([z[:0]])) == 0.0
    copy = torch.ones(3, device="cuda")
    assert zc.clip_grads([], 1.0, copies=[copy]).tolist() == [0.0, 1.0] and copy.tolist() == [1, 1, 1]
    one = torch.tensor([3.0, 4.0], device="cuda")
    assert zc.clip_grads([one], 5.0, eps=0.0).tolist() == [5.0, 1.0] and one.tolist() == [3.0, 4.0]
    assert zc.clip_grads([one], 0.0).tolist() == [5.0, 0.0] and one.tolist() == [0.0, 0.0]


def test_infinities_and_nan():
    a, b = grad(1, 9000, 1)[0], grad(30, 40, 2, dtype=torch.float32)
    a[77] = float("inf")
    assert zc.clip_grads([a, b], 1.0).tolist() == [float("inf"), 0.0]
    assert bool(torch.isnan(a[77])) and int(torch.isnan(a).sum()) == 1 and not bool(b.any())
    b[3, 4] = float("nan")
    r = zc.clip_grads([grad(1, 10, 3)[0], b], 1.0)
    assert bool(torch.isnan(r).all()) and bool(torch.isnan(b).all())


def test_sum_of_many_equal_squares():
    """Rounding errors that all point the same way stay within the bound."""
    g = torch.full((30_000_000,), 0.1, device="cuda")
    want = float(g[0].double()) * math.sqrt(g.numel())
    assert abs(float(zc.grad_norm([g])) - want) <= NORM * want


def test_same_bits_on_streams_and_in_graphs():
    grads = [grad(100, 777, 1), grad(3000, 1024, 2), grad(1, 5, 3, dtype=torch.float32)]
    start = [g.clone() for g in grads]
    clip = zc.GradClip(grads)
    want = clip.clip(0.25)
    scaled = [g.clone() for g in grads]

    def restore():
        for g, x in zip(grads, start):
            g.copy_(x)

    restore()
    assert torch.equal(clip.norm(), want[:1])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    r = clip.clip(0.25, stream=s)
    s.synchronize()
    assert torch.equal(r, want) and all(torch.equal(a, b) for a, b in zip(grads, scaled))
    restore()
    out = torch.empty(2, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        clip.clip(0.25, out=out)
    for k in range(3):
        restore()
        g.replay()
        assert torch.equal(out, want) and all(torch.equal(a, b) for a, b in zip(grads, scaled))


def test_executors_clip_each_parameter_once():
    """The reduced gradients of the three executors: a straddling parameter's
    copies are scaled and counted once, and nothing else is touched."""
    world, sizes = 4, np.array([700, 333, 1025, 64, 9, 2000, 31], np.int64)
    tree = workloads.Tree([f"p{i}" for i in range(len(sizes))], sizes)
    layout = workloads.arrival_layout(tree, capacity=None)
    buckets = [(b.start, b.tasks) for b in layout.buckets]
    rows = grad(world, tree.total, 1, dtype=torch.float32)
    mean = rows.double().mean(0)
    want = float(mean.norm())
    c = 0.5 * want / (want + 1e-6)

    ex = zc.Zero1Executor(world, sizes, layout.row_offset, buckets, torch.float32, fill=1e3)
    assert (ex.omap.owner < 0).any(), "a parameter straddles"
    ex.flush_all(rows)
    got = ex.grad_clip().clip(0.5 * want)
    assert abs(float(got[0]) - want) <= 1e-6 * want
    for r in range(world):
        slots = torch.zeros_like(ex.grad.buf[r], dtype=torch.bool)
        for p in range(len(sizes)):
            g = ex.grad.view(r, p)
            if g is None:
                continue
            o = int(layout.row_offset[p])
            assert torch.allclose(g.double(), mean[o:o + int(sizes[p])] * c, rtol=1e-5, atol=1e-9)
            slots[ex.grad.slot[r][p]:ex.grad.slot[r][p] + int(sizes[p])] = True
        assert bool((ex.grad.buf[r][~slots] == 1e3).all())

    part = zc.PartitionedExecutor(world, sizes, layout.row_offset, buckets, torch.float32)
    part.flush_all(rows)
    got = part.grad_clip().clip(0.5 * want)
    assert abs(float(got[0]) - want) <= 1e-6 * want
    flat = torch.cat([mean[int(layout.row_offset[p]):int(layout.row_offset[p]) + int(sizes[p])] for p in range(len(sizes))])
    assert torch.allclose(torch.cat(part.parts)[:tree.total].double(), flat * c, rtol=1e-5, atol=1e-9)

    own = rows.clone()
    inp = zc.InPlaceExecutor(world, sizes, buckets, torch.float32)
    inp.flush_all(own)
    got = inp.grad_clip(own).clip(0.5 * want)
    assert abs(float(got[0]) - want) <= 1e-6 * want
    for p in range(len(sizes)):
        o, e = int(layout.row_offset[p]), int(layout.row_offset[p]) + int(sizes[p])
        for r in range(world):
            if inp.omap.owner[p] in (-1, r):
                assert torch.allclose(own[r, o:e].double(), mean[o:e] * c, rtol=1e-5, atol=1e-9)
            else:
                assert torch.equal(own[r, o:e], rows[r, o:e])


def test_refusals():
    g = grad(10, 20, 1)
    keep = g.clone()
    with pytest.raises(zc.DpredError) as e:
        zc.clip_grads([g, g], 1e-9)
    assert e.value.code == -3 and torch.equal(g, keep)
    with pytest.raises(zc.DpredError):
        zc.clip_grads([g], 1e-9, copies=[g[3:4]])
    with pytest.raises(zc.DpredError):
        zc.clip_grads([g], -1.0)
    with pytest.raises(zc.DpredError):
        zc.clip_grads([g], 1.0, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(TypeError):
        zc.grad_norm([g.half()])
    with pytest.raises(ValueError):
        zc.grad_norm([g.cpu()])
    with pytest.raises(ValueError):
        zc.grad_norm([g.t()])
    with pytest.raises(ValueError):
        zc.grad_norm([g], out=torch.empty(2, device="cuda"))
    assert abs(float(zc.grad_norm([g, g])) - 2 ** 0.5 * norm64([g])) < 1e-5  # only reading, it may be named twice

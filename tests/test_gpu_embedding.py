"""The embedding and its gradient against 64-bit ones.

Tolerances.  Lookup: w * scale is one rounding in fp32 (2^-24) and one to the
output's type.  Gradient: a row of n tokens is summed in fp32 with at most n +
n / 32 + 9 additions (runs of up to 32 positions, then 8 shares of their sums), each
off by at most 2^-24 of the terms' magnitudes; the scale and the value added to
are one or two roundings more; one rounding to the output's type."""
import pytest
import torch

import zero_collectives_gb300 as zc

pytestmark = pytest.mark.gpu
BOUNDS = -7
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def randn(*shape, seed, scale=1.0, dtype=torch.bfloat16, pad=0, shift=0):
    """Rows of a wider tensor (pad) that starts `shift` elements into its storage."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rows, cols = shape
    t = (torch.randn(rows * (cols + pad) + shift, device="cuda", generator=g) * scale).to(dtype)
    return t[shift:].view(rows, cols + pad)[:, :cols]


def ids_of(t, v, seed, kind="uniform", dtype=torch.int64):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if kind == "one":
        i = torch.full((t,), v // 2, device="cuda")
    elif kind == "two":
        i = torch.where(torch.rand(t, device="cuda", generator=g) < 0.5, 0, v - 1)
    elif kind == "sorted":
        i = torch.arange(t, device="cuda") * v // max(t, 1)
    elif kind == "skewed":
        i = (torch.rand(t, device="cuda", generator=g) ** 6 * v).long().clamp_(0, v - 1)
    else:
        i = torch.randint(0, v, (t,), device="cuda", generator=g)
    return i.to(dtype)


@pytest.mark.parametrize("t,v,d", [(1, 1, 1), (1, 1000, 1024), (5, 7, 3), (33, 100, 64), (300, 500, 777), (1000, 40, 8), (4097, 3000, 256), (64, 50, 2056),
                                   (20000, 11, 16), (777, 60, 264), (3000, 90, 512), (300, 40, 5000)])
@pytest.mark.parametrize("wdt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("odt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pad,shift", [(0, 0), (8, 8), (3, 1)])
def test_embedding(t, v, d, wdt, odt, pad, shift):
    w = randn(v, d, seed=1, dtype=wdt, pad=pad, shift=shift)
    ids = ids_of(t, v, 2, dtype=torch.int32 if t % 2 else torch.int64)
    out = randn(t, d, seed=3, dtype=odt, pad=pad, shift=shift)
    gap = out.as_strided((max(t - 1, 1), pad), (d + pad, 1), out.storage_offset() + d).clone() if pad and t > 1 else None
    got = zc.embedding(ids, w, scale=1.7, out=out)
    scale = float(torch.tensor(1.7, dtype=torch.float32))
    want = w.double()[ids.long()] * scale
    assert bool(((got.double() - want).abs() <= (HALF[odt] + 2.0 ** -23) * want.abs()).all())
    if gap is not None:
        assert torch.equal(out.as_strided((t - 1, pad), (d + pad, 1), out.storage_offset() + d), gap), "columns between the rows were written"
    assert zc.device_status() == 0


def test_embedding_shapes_and_types():
    w = randn(20, 24, seed=1)
    ids = ids_of(12, 20, 2).view(3, 4)
    y = zc.embedding(ids, w)
    assert tuple(y.shape) == (3, 4, 24) and y.dtype is w.dtype and torch.equal(y, w[ids])
    assert torch.equal(zc.embedding(ids, w, out=torch.empty(12, 24, device="cuda")).view(3, 4, 24), w[ids].float())
    assert tuple(zc.embedding(ids[0, 0], w).shape) == (24,)
    assert tuple(zc.embedding(ids[:0], w).shape) == (0, 4, 24) and tuple(zc.embedding(ids, w[:, :0]).shape) == (3, 4, 0)
    dw = torch.empty(20, 24, device="cuda")
    zc.embedding_grad(ids, y, dw)
    assert torch.equal(dw, zc.embedding_grad(ids.view(-1), y.view(12, 24), torch.empty_like(dw)))


@pytest.mark.parametrize("id_type", [torch.int32, torch.int64])
def test_ids_outside_the_table(id_type):
    """They read and write nothing, and are reported; the others are not affected."""
    v, d = 100, 72
    w, dy = randn(v, d, seed=1), randn(6, d, seed=2, dtype=torch.float32)
    bad = torch.tensor([5, -1, 99, 100, 5, 2147483647], dtype=id_type, device="cuda")
    if id_type is torch.int64:
        bad[3] = (1 << 40) + 5
    y = zc.embedding(bad, w)
    assert zc.device_status(clear=True) == BOUNDS and zc.device_status() == 0
    assert torch.equal(y[[0, 2, 4]], w[[5, 99, 5]]) and not bool(y[[1, 3, 5]].any())
    for accumulate in (False, True):
        dw = randn(v, d, seed=3, dtype=torch.float32)
        want = dw.clone() if accumulate else torch.zeros_like(dw)
        zc.embedding_grad(bad, dy, dw, accumulate=accumulate)
        assert zc.device_status(clear=True) == BOUNDS
        want[5] = want[5] + (dy[0] + dy[4])
        want[99] = want[99] + dy[2]
        assert torch.equal(dw, want)
    zc.embedding_grad(torch.full((3,), 7, dtype=id_type, device="cuda"), dy[:3], torch.empty(v, d, device="cuda"), padding=7)
    assert zc.device_status() == 0


def check_grad(ids, dy, dw, scale, padding, accumulate):
    v, d = dw.shape
    before = dw.double() if accumulate else torch.zeros(v, d, dtype=torch.float64, device="cuda")
    keep = torch.ones_like(ids, dtype=torch.bool) if padding is None else ids != padding
    i, g = ids.long()[keep], dy.double()[keep]
    zc.embedding_grad(ids, dy, dw, scale=scale, padding=padding, accumulate=accumulate)
    scale = float(torch.tensor(scale, dtype=torch.float32))
    want = before + torch.zeros_like(before).index_add_(0, i, g) * scale
    mags = before.abs() + torch.zeros_like(before).index_add_(0, i, g.abs()) * abs(scale)
    n = torch.zeros(v, dtype=torch.float64, device="cuda").index_add_(0, i, torch.ones_like(i, dtype=torch.float64))[:, None]
    tol = HALF[dw.dtype] * want.abs() + (n * 33 / 32 + 12) * 2.0 ** -24 * mags
    bad = (dw.double() - want).abs() - tol
    assert bool(torch.isfinite(dw).all()) and float(bad.max()) <= 0, f"off by {float(bad.max()):.3g} beyond the tolerance"
    if not accumulate:
        assert not bool(dw[n[:, 0] == 0].any()), "a row without a token is not zero"
    else:
        assert torch.equal(dw[n[:, 0] == 0].double(), before[n[:, 0] == 0]), "a row without a token was written"
    assert zc.device_status() == 0


@pytest.mark.parametrize("t,v,d", [(1, 1, 1), (1, 1000, 1024), (2, 31, 8), (31, 5, 40), (32, 33, 64), (33, 100, 777), (65, 3, 256), (333, 1000, 264),
                                   (1000, 98304, 16), (4096, 20000, 520), (10000, 700, 72), (30001, 150, 33)])
@pytest.mark.parametrize("kind", ["uniform", "skewed", "one", "two", "sorted"])
@pytest.mark.parametrize("gdt,odt,accumulate", [(torch.bfloat16, torch.bfloat16, False), (torch.float32, torch.float32, True),
                                                (torch.bfloat16, torch.float32, False), (torch.float32, torch.bfloat16, True)])
def test_embedding_grad(t, v, d, kind, gdt, odt, accumulate):
    ids = ids_of(t, v, 5, kind, torch.int32 if t % 2 else torch.int64)
    dy, dw = randn(t, d, seed=1, dtype=gdt), randn(v, d, seed=2, dtype=odt)
    check_grad(ids, dy, dw, 0.3, v - 1 if t % 3 == 0 else None, accumulate)


@pytest.mark.parametrize("t,v", [(70001, 500), (65536, 40000), (65535, 3), (200000, 7)])
@pytest.mark.parametrize("kind", ["uniform", "skewed", "one"])
def test_many_tokens(t, v, kind):
    """Either side of what fits counters of 16 bits, and more tokens of a row than those hold."""
    check_grad(ids_of(t, v, 9, kind), randn(t, 8, seed=1), randn(v, 8, seed=2, dtype=torch.float32), 1.0, None, False)


@pytest.mark.parametrize("pad,shift", [(8, 0), (8, 8), (1, 0), (0, 1), (3, 5)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_embedding_grad_strides(pad, shift, accumulate):
    t, v, d = 500, 90, 136
    dy = randn(t, d, seed=1, pad=pad, shift=shift)
    dw = randn(v, d, seed=2, dtype=torch.float32, pad=pad, shift=shift)
    gap = dw.as_strided((v - 1, pad), (d + pad, 1), dw.storage_offset() + d).clone() if pad else None
    check_grad(ids_of(t, v, 3, "skewed"), dy, dw, 1.0, None, accumulate)
    if pad:
        assert torch.equal(dw.as_strided((v - 1, pad), (d + pad, 1), dw.storage_offset() + d), gap)


@pytest.mark.parametrize("v", [300, 200000, 300001])
def test_many_ids_per_block(v):
    """Tables of more rows than blocks times counters, and tokens at their ends."""
    ids = torch.tensor([0, v - 1, v - 1, v // 2, 0, v - 2] * 400, device="cuda")
    check_grad(ids, randn(2400, 24, seed=1), randn(v, 24, seed=2, dtype=torch.float32), 2.0, None, False)


def test_no_tokens():
    ids = torch.zeros(0, dtype=torch.int64, device="cuda")
    dy, dw = torch.zeros(0, 40, device="cuda"), randn(70, 40, seed=1)
    keep = dw.clone()
    assert torch.equal(zc.embedding_grad(ids, dy, dw, accumulate=True), keep)
    assert not bool(zc.embedding_grad(ids, dy, dw).any())
    only_padding = torch.full((100,), 3, device="cuda")
    assert torch.equal(zc.embedding_grad(only_padding, randn(100, 40, seed=2), keep.clone(), padding=3, accumulate=True), keep)
    assert not bool(zc.embedding_grad(only_padding, randn(100, 40, seed=2), dw.fill_(1.0), padding=3).any())


def test_special_values_stay_in_their_row():
    ids = torch.tensor([3, 4, 3, 5, 6], device="cuda").repeat(50)
    dy = randn(250, 64, seed=1)
    clean = zc.embedding_grad(ids, dy, torch.empty(9, 64, device="cuda"))
    dy[1, 5], dy[3, 6] = float("nan"), float("inf")
    got = zc.embedding_grad(ids, dy, torch.empty(9, 64, device="cuda"))
    assert bool(torch.isnan(got[4, 5])) and bool(torch.isinf(got[5, 6]))
    clean[4, 5], clean[5, 6] = got[4, 5], got[5, 6]
    assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(clean))


def test_same_bits_on_streams_and_in_graphs():
    t, v, d = 3000, 2000, 200
    ids, dy = ids_of(t, v, 1, "skewed"), randn(t, d, seed=2)
    w = randn(v, d, seed=3)
    dw = torch.zeros(v, d, device="cuda")
    want = zc.embedding_grad(ids, dy, dw).clone()
    look = zc.embedding(ids, w, scale=3.0)
    assert torch.equal(zc.embedding_grad(ids, dy, dw.fill_(1.0)), want)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got, out = torch.empty_like(dw), torch.empty_like(look)
    zc.embedding_grad(ids, dy, got, stream=s)
    zc.embedding(ids, w, scale=3.0, out=out, stream=s)
    s.synchronize()
    assert torch.equal(got, want) and torch.equal(out, look)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        zc.embedding_grad(ids, dy, got)
        zc.embedding(ids, w, scale=3.0, out=out)
    for seed in (7, 8):
        ids.copy_(ids_of(t, v, seed))
        dy.copy_(randn(t, d, seed=seed + 1))
        g.replay()
        assert torch.equal(got, zc.embedding_grad(ids, dy, torch.empty_like(dw))) and torch.equal(out, zc.embedding(ids, w, scale=3.0))


def test_gradient_against_differences():
    """The loss is linear in the table: a difference along a direction is the
    gradient itself, up to the gradient's own roundings."""
    t, v, d = 400, 60, 48
    ids, dy = ids_of(t, v, 1, "skewed"), randn(t, d, seed=2)
    dw = zc.embedding_grad(ids, dy, torch.empty(v, d, device="cuda"), scale=1.5)
    w, step = randn(v, d, seed=3).double(), randn(v, d, seed=4).double()

    def loss(x):
        return (dy.double() * x[ids] * 1.5).sum()

    diff = (loss(w + 0.5 * step) - loss(w - 0.5 * step))
    mags = torch.zeros(v, d, dtype=torch.float64, device="cuda").index_add_(0, ids, dy.double().abs()) * 1.5
    assert abs(float((dw.double() * step).sum() - diff)) <= (t + 16) * 2.0 ** -24 * float((mags * step.abs()).sum())


def test_refusals():
    w, ids = randn(10, 8, seed=1), torch.zeros(4, dtype=torch.int64, device="cuda")
    dy, dw = randn(4, 8, seed=2), torch.zeros(10, 8, device="cuda")
    with pytest.raises(TypeError):
        zc.embedding(ids.float(), w)
    with pytest.raises(TypeError):
        zc.embedding(ids, w.half())
    with pytest.raises(ValueError):
        zc.embedding(torch.zeros(4, 2, dtype=torch.int64, device="cuda")[:, 0], w)
    with pytest.raises(ValueError):
        zc.embedding(ids.cpu(), w)
    with pytest.raises(ValueError):
        zc.embedding(ids, w.t())
    with pytest.raises(ValueError):
        zc.embedding(ids, w, out=torch.empty(5, 8, device="cuda"))
    with pytest.raises(ValueError):
        zc.embedding_grad(ids, dy[:3], dw)
    with pytest.raises(ValueError):
        zc.embedding_grad(ids, dy, dw, padding=10)
    with pytest.raises(ValueError):
        zc.embedding_grad(ids, dy, dw, padding=-1)
    with pytest.raises(ValueError):
        zc.embedding_grad(ids, dy, torch.zeros(10, 9, device="cuda"))
    with pytest.raises(zc.DpredError):
        zc.embedding_grad(ids, dy, dw, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(zc.DpredError):
        zc.embedding(ids, w, scale=float("inf"))
    assert not bool(dw.any())

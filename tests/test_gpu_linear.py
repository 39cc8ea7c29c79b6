"""Linear-layer products against plain 64-bit ones.

Tolerance of an element, derived from the arithmetic: products of bf16 values
are exact in fp32; a sum of K terms in fp32 is off by at most K 2^-23 times the
sum of the terms' magnitudes (2^-23: a unit in the last place, which covers
truncation as well as rounding); the activations have slopes below 1.2 and
their exponential and reciprocal are good to 2^-18 of |z| + 1; one rounding to
bf16 adds 2^-8 of the value (fp32: 2^-23)."""
import math

import pytest
import torch

import zero_collectives_gb300 as zc

pytestmark = pytest.mark.gpu
ACTS = ("none", "relu", "gelu", "silu")


def randn(*shape, seed, scale=1.0, dtype=torch.bfloat16, pad=0, shift=0):
    """Rows of a wider tensor (pad) that starts `shift` elements into its storage."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rows, cols = shape
    t = (torch.randn(rows * (cols + pad) + shift, device="cuda", generator=g) * scale).to(dtype)
    return t[shift:].view(rows, cols + pad)[:, :cols]


def act64(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if act == "silu":
        return z * torch.sigmoid(z)
    return z


def act_grad64(z, act):
    z = z.detach().clone().requires_grad_(True)
    return torch.autograd.grad(act64(z, act).sum(), z)[0] if act != "none" else torch.ones_like(z)


def close(got, want, mags, terms, slack=0.0):
    """mags: sum of the terms' magnitudes; terms: how many of them."""
    last = 2.0 ** -8 if got.dtype == torch.bfloat16 else 2.0 ** -23
    tol = last * want.abs() + 1.2 * (terms + 4) * 2.0 ** -23 * mags + slack
    bad = (got.double() - want).abs() - tol
    assert bool(torch.isfinite(got).all())
    assert float(bad.max()) <= 0, f"off by {float(bad.max()):.3g} beyond the tolerance"


SHAPES = [(1, 64, 64), (1, 4096, 1024), (1, 1, 1), (3, 5, 7), (7, 129, 63), (33, 200, 65), (64, 512, 512),
          (65, 96, 2048), (128, 128, 64), (129, 257, 130), (333, 1000, 777), (512, 640, 320), (1000, 24, 4000),
          (1024, 2048, 512), (2500, 1300, 96)]


@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("act", ACTS)
def test_linear(m, n, k, act):
    x, w = randn(m, k, seed=1), randn(n, k, seed=2, scale=1 / math.sqrt(k))
    b = randn(1, n, seed=3, dtype=torch.float32 if m % 2 else torch.bfloat16)[0]
    r = randn(m, n, seed=4)
    z = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
    y = zc.linear(x, w, bias=b, act=act, residual=r, preact=z)
    z64 = x.double() @ w.double().T + b.double()
    mags = x.double().abs() @ w.double().abs().T + b.double().abs()
    close(z, z64, mags, k)
    close(y, act64(z64, act) + r.double(), mags + r.double().abs(), k, 2.0 ** -18 * (z64.abs() + 1))
    assert zc.device_status() == 0


@pytest.mark.parametrize("m", [1, 40, 300])
@pytest.mark.parametrize("pad,shift", [(8, 0), (8, 8), (1, 0), (0, 1), (3, 5)])
def test_linear_strides_and_alignment(m, pad, shift):
    n, k = 136, 200
    x, w = randn(m, k, seed=1, pad=pad, shift=shift), randn(n, k, seed=2, pad=pad, shift=shift)
    r = randn(m, n, seed=4, pad=pad, shift=shift)
    out = randn(m, n, seed=5, pad=pad, shift=shift, dtype=torch.float32)
    hold = out.as_strided((m, n + pad), (n + pad, 1), out.storage_offset()) if m == 1 or pad == 0 else \
        out.as_strided((m - 1, n + pad), (n + pad, 1), out.storage_offset())
    before = hold[:, n:].clone()
    y = zc.linear(x, w, residual=r, out=out)
    assert y.data_ptr() == out.data_ptr()
    want = x.double() @ w.double().T + r.double()
    close(y, want, x.double().abs() @ w.double().abs().T + r.double().abs(), k)
    assert torch.equal(hold[:, n:], before), "columns between the rows were written"


@pytest.mark.parametrize("m,n,k", [(0, 8, 8), (8, 0, 8), (5, 6, 0), (100, 70, 0)])
def test_linear_empty(m, n, k):
    x, w = torch.zeros(m, k, dtype=torch.bfloat16, device="cuda"), torch.zeros(n, k, dtype=torch.bfloat16, device="cuda")
    b = randn(1, n, seed=3)[0] if n else torch.zeros(0, dtype=torch.bfloat16, device="cuda")
    y = zc.linear(x, w, bias=b, act="relu")
    assert tuple(y.shape) == (m, n)
    assert torch.equal(y, b.clamp(min=0).expand(m, n))


def test_linear_special_values():
    """A NaN or an infinity reaches its own row only; padding never leaks into a result."""
    m, n, k = 70, 72, 100
    x, w = randn(m, k, seed=1), randn(n, k, seed=2)
    clean = zc.linear(x, w, act="silu")
    x2 = x.clone()
    x2[3, 99] = float("nan")
    x2[5, 0] = float("inf")
    y = zc.linear(x2, w, act="silu")
    keep = [i for i in range(m) if i not in (3, 5)]
    assert torch.equal(y[keep], clean[keep])
    assert bool(torch.isnan(y[3]).all()) and not bool(torch.isfinite(y[5].float()).all())
    z = torch.tensor([[-3e38, -1e20, -100.0, 100.0, 1e20, 3e38, 0.0, -0.0]], device="cuda").bfloat16()
    dy = torch.ones(1, 8, dtype=torch.bfloat16, device="cuda")
    eye = torch.eye(8, dtype=torch.bfloat16, device="cuda")
    for act in ("gelu", "silu", "relu"):
        g = zc.linear_dgrad(dy, eye, preact=z, act=act)
        half = 0.0 if act == "relu" else 0.5
        assert torch.equal(g.float().cpu(), torch.tensor([[0, 0, 0, 1, 1, 1, half, half]])), act


@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("act", ACTS)
def test_linear_dgrad(m, n, k, act):
    dy, w = randn(m, n, seed=1), randn(n, k, seed=2, scale=1 / math.sqrt(n))
    r, z = randn(m, k, seed=3), randn(m, k, seed=4, scale=2.0)
    dx = zc.linear_dgrad(dy, w, preact=z, act=act, residual=r)
    g = act_grad64(z.double(), act)
    want = (dy.double() @ w.double() + r.double()) * g
    mags = dy.double().abs() @ w.double().abs() + r.double().abs()
    close(dx, want, mags, n, 2.0 ** -18 * mags * (z.double().abs() + 1))


@pytest.mark.parametrize("pad,shift", [(8, 0), (1, 0), (3, 5)])
@pytest.mark.parametrize("m", [2, 200])
def test_linear_dgrad_strides(m, pad, shift):
    n, k = 200, 136
    dy, w = randn(m, n, seed=1, pad=pad, shift=shift), randn(n, k, seed=2, pad=pad, shift=shift)
    z = randn(m, k, seed=4, pad=pad, shift=shift)
    dx = zc.linear_dgrad(dy, w, preact=z, act="gelu", out_dtype=torch.float32)
    mags = dy.double().abs() @ w.double().abs()
    close(dx, dy.double() @ w.double() * act_grad64(z.double(), "gelu"), mags, n, 2.0 ** -18 * mags * (z.double().abs() + 1))


@pytest.mark.parametrize("m,n,k", SHAPES + [(20000, 72, 40), (4097, 128, 256)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("accumulate", [False, True])
def test_linear_wgrad(m, n, k, dtype, accumulate):
    dy, x = randn(m, n, seed=1), randn(m, k, seed=2)
    dw, db = randn(n, k, seed=3, dtype=dtype), randn(1, n, seed=4, dtype=torch.float32)[0]
    dw0, db0 = dw.double() * accumulate, db.double() * accumulate
    zc.linear_wgrad(dy, x, dw, bias_grad=db, accumulate=accumulate)
    close(dw, dy.double().T @ x.double() + dw0, dy.double().abs().T @ x.double().abs() + dw0.abs(), m)
    close(db, dy.double().sum(0) + db0, dy.double().abs().sum(0) + db0.abs(), m)
    assert zc.device_status() == 0


@pytest.mark.parametrize("m,n,k", [(1500, 700, 1000), (700, 4000, 1100), (640, 72, 5000), (333, 333, 2100), (6000, 1024, 1024), (64, 2048, 4096)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pad,accumulate", [(0, False), (3, True)])
def test_bias_gradient_beside_many_tiles(m, n, k, dtype, pad, accumulate):
    """Every column of dy counts once, whatever kernel sums it, and a repeated call has the same bits."""
    dy, x = randn(m, n, seed=1, pad=pad), randn(m, k, seed=2)
    dw0, db0 = randn(n, k, seed=3, dtype=dtype), randn(1, n, seed=4, dtype=torch.float32)[0]
    got = []
    for want_db in (True, True, False):
        dw, db = dw0.clone(), db0.clone()
        zc.linear_wgrad(dy, x, dw, bias_grad=db if want_db else None, accumulate=accumulate)
        got.append((dw, db))
    close(got[0][1], dy.double().sum(0) + db0.double() * accumulate, dy.double().abs().sum(0) + db0.double().abs() * accumulate, m)
    for dw, _ in got:
        close(dw, dy.double().T @ x.double() + dw0.double() * accumulate,
              dy.double().abs().T @ x.double().abs() + dw0.double().abs() * accumulate, m)
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1]) and torch.equal(got[2][1], db0)
    assert zc.device_status() == 0


@pytest.mark.parametrize("m,n,k,shift", [(5000, 5000, 520, 0), (5000, 5008, 520, 8), (4999, 5024, 1000, 16), (9000, 4500, 512, 0)])
@pytest.mark.parametrize("act", ["none", "silu"])
def test_long_reductions_over_many_ragged_tiles(m, n, k, shift, act):
    """Every element of a ragged output is written once, and nothing around it."""
    x, w = randn(m, k, seed=1), randn(n, k, seed=2, scale=1 / math.sqrt(k))
    flat = torch.full((m * n + shift + 64,), float("nan"), dtype=torch.bfloat16, device="cuda")
    y = zc.linear(x, w, act=act, out=flat[shift:shift + m * n].view(m, n))
    for rows in (slice(0, 300), slice(m - 300, m)):
        z = x[rows].double() @ w.double().T
        mags = x[rows].double().abs() @ w.double().abs().T
        close(y[rows], act64(z, act), mags, k, 2.0 ** -18 * mags)
    assert bool(torch.isfinite(y.float()).all())
    assert bool(torch.isnan(flat[:shift]).all()) and bool(torch.isnan(flat[shift + m * n:]).all())


def test_wgrad_into_gradient_rows():
    """Gradients land in the [W, n] row a flush reads, at an odd offset, and nothing else is touched."""
    m, n, k, off = 300, 40, 56, 13
    rows = torch.full((2, off + n * k + 9), float("nan"), dtype=torch.bfloat16, device="cuda")
    dy, x = randn(m, n, seed=1), randn(m, k, seed=2)
    zc.linear_wgrad(dy, x, rows[1, off:off + n * k].view(n, k))
    close(rows[1, off:off + n * k].view(n, k), dy.double().T @ x.double(), dy.double().abs().T @ x.double().abs(), m)
    assert bool(torch.isnan(rows[0]).all()) and bool(torch.isnan(rows[1, :off]).all()) and bool(torch.isnan(rows[1, off + n * k:]).all())


def test_wgrad_of_no_tokens():
    dy, x = torch.zeros(0, 24, dtype=torch.bfloat16, device="cuda"), torch.zeros(0, 40, dtype=torch.bfloat16, device="cuda")
    dw, db = randn(24, 40, seed=1, dtype=torch.float32), randn(1, 24, seed=2, dtype=torch.float32)[0]
    dw0, db0 = dw.clone(), db.clone()
    zc.linear_wgrad(dy, x, dw, bias_grad=db, accumulate=True)
    assert torch.equal(dw, dw0) and torch.equal(db, db0)
    zc.linear_wgrad(dy, x, dw, bias_grad=db)
    assert not bool(dw.any()) and not bool(db.any())


@pytest.mark.parametrize("act", ["relu", "gelu", "silu"])
def test_gradients_against_differences(act):
    """Backward of a two-layer block against central differences of its 64-bit
    forward along random directions.  The kernels' gradients carry bf16
    roundings of the stored z and of dz (2^-8 each, plus the result's own), so
    a directional derivative is off by at most 3 2^-8 of the sum of its terms'
    magnitudes; the differences' own error (h^2) is far below that."""
    m, d, f = 48, 40, 72
    x, w1, w2 = randn(m, d, seed=1), randn(f, d, seed=2, scale=0.2), randn(d, f, seed=3, scale=0.2)
    b1, dy = randn(1, f, seed=4, dtype=torch.float32)[0], randn(m, d, seed=5)
    z = torch.empty(m, f, dtype=torch.bfloat16, device="cuda")
    h = zc.linear(x, w1, bias=b1, act=act, preact=z)
    dz = zc.linear_dgrad(dy, w2, preact=z, act=act)
    dw2 = torch.empty(d, f, dtype=torch.float32, device="cuda")
    zc.linear_wgrad(dy, h, dw2)
    dw1, db1 = torch.empty(f, d, dtype=torch.float32, device="cuda"), torch.empty(f, dtype=torch.float32, device="cuda")
    zc.linear_wgrad(dz, x, dw1, bias_grad=db1)
    dx = zc.linear_dgrad(dz, w1, residual=dy)

    def loss(x, w1, b1, w2):
        return (dy.double() * (act64(x @ w1.T + b1, act) @ w2.T + x)).sum()

    at = [t.double() for t in (x, w1, b1, w2)]
    for i, grad in enumerate((dx, dw1, db1, dw2)):
        g = torch.Generator(device="cuda").manual_seed(20 + i)
        v = torch.randn(at[i].shape, device="cuda", generator=g, dtype=torch.float64)
        hs = 1e-5
        up, down = [list(at), list(at)]
        up[i], down[i] = at[i] + hs * v, at[i] - hs * v
        diff = (loss(*up) - loss(*down)) / (2 * hs)
        got = (grad.double() * v).sum()
        # relu has kinks at z = 0, where z's rounding may also pick the other side
        assert abs(float(got - diff)) <= 3 * 2.0 ** -8 * float((grad.double() * v).abs().sum())


def test_streams_and_graph():
    """Calls on a side stream and inside a captured graph give the bits of plain calls."""
    m, n, k = 96, 160, 77  # k is odd: the operands are packed into a workspace
    x, w = randn(m, k, seed=1), randn(n, k, seed=2)
    want = zc.linear(x, w, act="gelu")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = zc.linear(x, w, act="gelu", stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    out = torch.zeros_like(want)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        zc.linear(x, w, act="gelu", out=out, workspace=ws)
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    x.copy_(randn(m, k, seed=9))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, zc.linear(x, w, act="gelu"))


def test_packed_operands_from_several_threads_and_streams():
    """Unaligned operands are packed into memory that no other thread or stream uses at the same time."""
    import threading
    m, n, k = 300, 200, 777
    cases = [(randn(m + i, k, seed=10 + i), randn(n, k, seed=20 + i)) for i in range(4)]
    want = [zc.linear(x, w) for x, w in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [[] for _ in cases]

    def work(i):
        x, w = cases[i]
        for _ in range(20):
            got[i].append(zc.linear(x, w, stream=streams[i % 2]))  # two threads share a stream

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(cases))]
    [t.start() for t in threads]
    [t.join() for t in threads]
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[i]) for i in range(len(cases)) for y in got[i])


def test_output_offsets_beyond_32_bits():
    m, n, k = 22000, 98304, 64   # 2.16e9 outputs
    x, w = randn(m, k, seed=1), randn(n, k, seed=2)
    y = zc.linear(x, w)
    for rows in (slice(0, 3), slice(10921, 10925), slice(m - 3, m)):
        close(y[rows], x[rows].double() @ w.double().T, x[rows].double().abs() @ w.double().abs().T, k)


@pytest.mark.parametrize("m,n,k", [(4096, 8192, 64), (2100, 16000, 64), (5000, 3900, 128), (16000, 2056, 192)])
@pytest.mark.parametrize("form", ["plain", "act", "pre", "residual", "all", "grad", "f32", "f32 add"])
def test_many_short_tiles(m, n, k, form):
    """Reductions so short that every tile's epilogue overtakes the copies of the one before."""
    x, w, b = randn(m, k, seed=1), randn(n, k, seed=2, scale=1 / math.sqrt(k)), randn(1, n, seed=3)[0]
    z64 = x.double() @ w.double().T
    mags = x.double().abs() @ w.double().abs().T
    if form in ("plain", "f32", "f32 add"):
        if form == "f32 add":  # the same product as a weight gradient added to an accumulator
            out = randn(m, n, seed=4, dtype=torch.float32)
            want = out.double() + z64
            zc.linear_wgrad(x.T.contiguous(), w.T.contiguous(), out, accumulate=True)
            return close(out, want, mags + want.abs(), k)
        return close(zc.linear(x, w, out_dtype=torch.float32 if form == "f32" else None), z64, mags, k)
    if form == "grad":
        z = randn(m, n, seed=5)
        dx = zc.linear_dgrad(x, w.T.contiguous(), preact=z, act="gelu")
        return close(dx, z64 * act_grad64(z.double(), "gelu"), mags, k, 2.0 ** -18 * mags * (z.double().abs() + 1))
    z64, mags = z64 + b.double(), mags + b.double().abs()
    r = randn(m, n, seed=4) if form in ("residual", "all") else None
    z = torch.empty(m, n, dtype=torch.bfloat16, device="cuda") if form in ("pre", "all") else None
    act = "none" if form == "residual" else "silu"
    y = zc.linear(x, w, bias=b, act=act, residual=r, preact=z)
    r64 = r.double() if r is not None else torch.zeros_like(z64)
    close(y, act64(z64, act) + r64, mags + r64.abs(), k, 2.0 ** -18 * (z64.abs() + 1))
    if z is not None:
        close(z, z64, mags, k)


def test_residual_in_place():
    m, n, k = 200, 264, 128
    x, w, r = randn(m, k, seed=1), randn(n, k, seed=2), randn(m, n, seed=3)
    want = zc.linear(x, w, residual=r)
    zc.linear(x, w, residual=r, out=r)
    assert torch.equal(r, want)

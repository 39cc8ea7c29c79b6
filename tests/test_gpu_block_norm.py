"""Norms, gate and residual sum between two blocks, and their gradients, against
64-bit ones.

Tolerances, in units of e = 2^-24 relative to the magnitudes of the terms.  A sum
over a row adds at most 32 fused steps of a thread, 5 of a warp and 16 warps: 53 e;
the mean and eps add 2 e, the root halves that, and the reciprocal root itself is
good to 2 units in the last place (4 e): i_y and i_r are within 32 e, n_y and n_r
within 33 e, gate u within 35 e, r within 36 e of its terms before its rounding.
Where r is off by a vector of relative length t, i_r is off by t as well.
Gradients: a mean of products with n adds 53 + 33 + 2 e, the product with i n 65 e,
the rest a few: g within 256 e = 2^-16 of the sum of its terms' magnitudes, and dy
within twice that of its own; a sum over m rows adds m e (and 64 for the way it is
split).  Each output then has its one rounding."""

import pytest
import torch

import zero_collectives_gb300 as zc

pytestmark = pytest.mark.gpu
E = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: E}


def randn(*shape, seed, scale=1.0, shift_value=0.0, dtype=torch.bfloat16, pad=0, shift=0):
    """Rows of a wider tensor (pad) that starts `shift` elements into its storage."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rows, cols = shape
    t = (torch.randn(rows * (cols + pad) + shift, device="cuda", generator=g) * scale + shift_value).to(dtype)
    return t[shift:].view(rows, cols + pad)[:, :cols]


class Case:
    """Inputs of a call, and the formulas in 64 bits."""

    def __init__(self, m, d, stream=torch.bfloat16, y=True, post=True, gate=1, pre=True, scale=0.7, weights=torch.float32, dr=True, pad=0, shift=0,
                 eps=1e-6):
        kw = dict(pad=pad, shift=shift)
        self.m, self.d, self.eps = m, d, eps
        self.scale = scale if y else 1.0
        self.x = randn(m, d, seed=1, scale=2.0, dtype=stream, **kw)
        self.y = randn(m, d, seed=2, **kw) if y else None
        self.post = randn(1, d, seed=3, scale=0.2, shift_value=1.0, dtype=weights)[0] if y and post else None
        self.gate = randn(gate, d, seed=4, scale=0.3, shift_value=0.5, dtype=weights) if y and gate else None
        self.pre = randn(1, d, seed=5, scale=0.2, shift_value=1.0, dtype=weights)[0] if pre else None
        self.dr = randn(m, d, seed=6, scale=1e-2, dtype=stream, **kw) if dr else None
        self.dh = randn(m, d, seed=7, scale=1e-2, **kw) if pre else None
        self.s32 = float(torch.tensor(self.scale, dtype=torch.float32))
        self.e32 = float(torch.tensor(eps, dtype=torch.float32))

    def rows(self, gate):
        return gate.double().repeat_interleave(self.m // gate.shape[0], 0)

    def inv(self, a):
        return (a.square().mean(-1, keepdim=True) + self.e32).rsqrt()

    def forward(self, **kw):
        return zc.block_norm(self.x, y=self.y, post=self.post, gate=self.gate, residual_scale=self.scale, pre=self.pre, eps=self.eps, **kw)

    def check_forward(self, r, h):
        want = self.x.double()
        off = torch.zeros_like(want)
        if self.y is not None:
            u = self.y.double()
            if self.post is not None:
                u = u * self.inv(u) * self.post.double()
            if self.gate is not None:
                u = u * self.rows(self.gate)
            want, off = self.s32 * want + u, 36 * E * ((self.s32 * want).abs() + u.abs())
            assert r.dtype is self.x.dtype
            near(r, want, off)
        if self.pre is None:
            assert h is None
            return
        i = self.inv(want)
        n = want * i * self.pre.double()
        t = off.norm(dim=-1, keepdim=True) / want.norm(dim=-1, keepdim=True).clamp(min=1e-300)
        near(h, n, n.abs() * (36 * E + t) + i * self.pre.double().abs() * off)

    def grads(self, dtype=torch.float32, fill=0.0):
        def like(w):
            return None if w is None else torch.full(w.shape, fill, dtype=dtype, device="cuda")
        return dict(post_grad=like(self.post), gate_grad=like(self.gate), pre_grad=like(self.pre))

    def backward(self, grads, accumulate=False, **kw):
        return zc.block_norm_grad(self.x, dr=self.dr, dh=self.dh, y=self.y, post=self.post, gate=self.gate, residual_scale=self.scale, pre=self.pre,
                                  eps=self.eps, accumulate=accumulate, **grads, **kw)

    def check_backward(self, dx, dy, grads, fill=0.0):
        r, m = self.x.double(), self.m
        zero = torch.zeros_like(r)
        g, gm = (zero, zero) if self.dr is None else (self.dr.double(), self.dr.double().abs())

        def weight(got, want, mags, slack):
            near(got, want + fill, slack + (m + 64) * E * (mags + abs(fill)))

        if self.pre is not None:
            i, dh, w = self.inv(r), self.dh.double(), self.pre.double()
            n, v = r * i, dh * w
            if grads["pre_grad"] is not None:
                weight(grads["pre_grad"], (dh * n).sum(0), (dh * n).abs().sum(0), 36 * E * (dh * n).abs().sum(0))
            g = g + i * (v - n * (v * n).mean(-1, keepdim=True))
            gm = gm + i * (v.abs() + n.abs() * (v * n).abs().mean(-1, keepdim=True))
        near(dx, self.s32 * g, 2.0 ** -16 * abs(self.s32) * gm)
        if self.y is None:
            assert dy is None
            return
        y = self.y.double()
        i = self.inv(y) if self.post is not None else torch.ones_like(y[:, :1])
        n = y * i
        if self.gate is not None:
            u = n * self.post.double() if self.post is not None else n
            if grads["gate_grad"] is not None:
                k = self.gate.shape[0]
                mags = (gm * u.abs()).view(k, m // k, -1).sum(1)
                weight(grads["gate_grad"], (g * u).view(k, m // k, -1).sum(1), mags, 2.0 ** -15 * mags)
            g, gm = g * self.rows(self.gate), gm * self.rows(self.gate).abs()
        if self.post is not None:
            if grads["post_grad"] is not None:
                weight(grads["post_grad"], (g * n).sum(0), (gm * n.abs()).sum(0), 2.0 ** -15 * (gm * n.abs()).sum(0))
            g, gm = g * self.post.double(), gm * self.post.double().abs()
            g = i * (g - n * (g * n).mean(-1, keepdim=True))
            gm = i * (gm + n.abs() * (gm * n.abs()).mean(-1, keepdim=True))
        near(dy, g, 2.0 ** -15 * gm)


def near(got, want, tol):
    bad = (got.double() - want).abs() - HALF[got.dtype] * want.abs() * (1 + 2.0 ** -8) - tol * (1 + 2.0 ** -7)
    assert bool(torch.isfinite(got).all()) and float(bad.max()) <= 0, f"off by {float(bad.max()):.3g} beyond the tolerance"


SIZES = [(1, 1), (1, 8), (1, 1024), (3, 5), (7, 31), (33, 64), (64, 72), (300, 256), (257, 264), (130, 777), (1000, 512), (2000, 1024), (70, 2048),
         (65, 4096), (40, 4104), (33, 8192), (21, 12288), (9, 16384), (5, 16383), (20, 5001), (6000, 96)]
FORMS = [dict(), dict(gate=0), dict(post=False), dict(post=False, gate=0), dict(pre=False), dict(post=False, pre=False), dict(y=False),
         dict(pre=False, gate=0)]


@pytest.mark.parametrize("m,d", SIZES)
@pytest.mark.parametrize("stream,weights", [(torch.bfloat16, torch.float32), (torch.float32, torch.bfloat16)])
@pytest.mark.parametrize("form", FORMS, ids=str)
def test_both_directions(m, d, stream, weights, form):
    c = Case(m, d, stream=stream, weights=weights, **form)
    c.check_forward(*c.forward())
    grads = c.grads(fill=0.25)
    dx, dy = c.backward(grads)
    c.check_backward(dx, dy, grads)
    assert zc.device_status() == 0


@pytest.mark.parametrize("m,d", [(1, 64), (12, 200), (600, 264), (6000, 128), (1200, 1024), (24, 4104), (30, 777)])
@pytest.mark.parametrize("stream", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("share", ["token", "two", "few", "three", "half"])
def test_gates_of_sequences_and_tokens(m, d, stream, share):
    k = {"token": m, "two": 2, "few": max(1, m // 12), "three": 3, "half": max(1, m // 2)}[share]
    k = k if m % k == 0 else 1
    c = Case(m, d, stream=stream, gate=k)
    c.check_forward(*c.forward())
    grads = c.grads(fill=-0.5)
    dx, dy = c.backward(grads, accumulate=True)
    c.check_backward(dx, dy, grads, fill=-0.5)


# rows enough for every row group to have several, at each width's way of covering a row
MANY = [(9000, 33), (9001, 64), (9000, 250), (6000, 400), (6000, 509), (6000, 777), (5500, 1000), (3000, 1537), (3001, 2048), (1500, 3333), (1400, 4096),
        (900, 5001), (801, 8192), (700, 8191), (500, 12288), (500, 12289), (420, 16384), (420, 16383)]


@pytest.mark.parametrize("m,d", MANY)
@pytest.mark.parametrize("stream", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("form", [dict(), dict(gate="token"), dict(y=False), dict(post=False, gate=0, dr=False)], ids=str)
def test_many_rows(m, d, stream, form):
    form = dict(form)
    if form.get("gate") == "token":
        form["gate"] = m
    c = Case(m, d, stream=stream, **form)
    c.check_forward(*c.forward())
    grads = c.grads(fill=0.125)
    dx, dy = c.backward(grads, accumulate=True)
    c.check_backward(dx, dy, grads, fill=0.125)
    assert zc.device_status() == 0


@pytest.mark.parametrize("m,d,pad,shift", [(6000, 97, 0, 1), (6000, 1, 0, 3), (6001, 3, 2, 1), (20000, 5, 0, 7), (5000, 1024, 1, 0), (5000, 1000, 3, 5), (1000, 5000, 0, 1),
                                          (400, 16000, 7, 3)])
@pytest.mark.parametrize("stream", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("gate", [1, 4, 0])
def test_many_rows_of_any_alignment(m, d, pad, shift, stream, gate):
    """Rows that share 16-byte pieces with their neighbours, shorter than a piece, and
    at the ends of their storage; into outputs whose gaps stay as they are."""
    gate = gate if gate == 0 or m % gate == 0 else m
    c = Case(m, d, stream=stream, gate=gate, pad=pad, shift=shift)
    outs = [randn(m, d, seed=20 + i, dtype=t, pad=pad, shift=shift) for i, t in enumerate((stream, torch.bfloat16, stream, torch.bfloat16))]
    gaps = [o.as_strided((m - 1, pad), (d + pad, 1), o.storage_offset() + d) for o in outs]
    before = [g.clone() for g in gaps]
    c.check_forward(*c.forward(out=outs[0], out_norm=outs[1]))
    grads = c.grads()
    c.check_backward(*c.backward(grads, dx=outs[2], dy=outs[3]), grads)
    assert all(torch.equal(a, b) for a, b in zip(gaps, before)), "columns between the rows were written"
    # in place, over the rows themselves
    want = [o.clone() for o in outs]
    r2, h2 = c.forward(out=c.x, out_norm=c.y)
    assert torch.equal(r2, want[0]) and torch.equal(h2, want[1])
    k = Case(m, d, stream=stream, gate=gate, pad=pad, shift=shift)
    dx2, dy2 = k.backward(k.grads(), dx=k.dr, dy=k.dh)
    assert torch.equal(dx2, want[2]) and torch.equal(dy2, want[3])


@pytest.mark.parametrize("pad,shift", [(8, 0), (8, 8), (1, 0), (0, 1), (3, 5)])
@pytest.mark.parametrize("m,d", [(50, 136), (9, 2056)])
@pytest.mark.parametrize("stream", [torch.bfloat16, torch.float32])
def test_strides_and_alignment(m, d, pad, shift, stream):
    c = Case(m, d, stream=stream, pad=pad, shift=shift, gate=m if m % 2 else 2)
    outs = [randn(m, d, seed=20 + i, dtype=t, pad=pad, shift=shift) for i, t in enumerate((stream, torch.bfloat16, stream, torch.bfloat16))]
    gaps = [o.as_strided((m - 1, pad), (d + pad, 1), o.storage_offset() + d) for o in outs]
    before = [g.clone() for g in gaps]
    r, h = c.forward(out=outs[0], out_norm=outs[1])
    assert r is outs[0] and h is outs[1]
    c.check_forward(r, h)
    grads = c.grads(torch.bfloat16)
    grads["post_grad"] = None  # not every one is wanted
    dx, dy = c.backward(grads, dx=outs[2], dy=outs[3])
    c.check_backward(dx, dy, grads)
    assert all(torch.equal(a, b) for a, b in zip(gaps, before)), "columns between the rows were written"


@pytest.mark.parametrize("d", [96, 1024, 777])
def test_weight_gradients_in_either_type(d):
    for dtype in (torch.bfloat16, torch.float32):
        for accumulate in (False, True):
            c = Case(700, d, gate=7)
            grads = c.grads(dtype, fill=0.5)
            dx, dy = c.backward(grads, accumulate=accumulate)
            c.check_backward(dx, dy, grads, fill=0.5 * accumulate)


def test_no_gradient_from_above_or_none_wanted():
    c = Case(200, 264, dr=False)
    grads = c.grads()
    c.check_backward(*c.backward(grads), grads)
    c = Case(200, 264)
    nothing = dict(post_grad=None, gate_grad=None, pre_grad=None)
    c.check_backward(*c.backward(nothing), nothing)


@pytest.mark.parametrize("m", [1, 5, 3000])
@pytest.mark.parametrize("d", [72, 1024, 333, 8200])
def test_in_place(m, d):
    """r over x, h over y, dx over dr, dy over dh or y: the same bits."""
    c = Case(m, d)
    r, h = c.forward()
    x, y = c.x.clone(), c.y.clone()
    r2, h2 = zc.block_norm(x, y=y, post=c.post, gate=c.gate, residual_scale=c.scale, pre=c.pre, out=x, out_norm=y)
    assert r2 is x and torch.equal(x, r) and torch.equal(y, h)
    g = c.grads()
    dx, dy = c.backward(g)
    for over in ("dh", "y"):
        k = Case(m, d)
        g2 = k.grads()
        dx2, dy2 = k.backward(g2, dx=k.dr, dy=getattr(k, over))
        assert torch.equal(dx2, dx) and torch.equal(dy2, dy) and all(torch.equal(g[n], g2[n]) for n in g)


def test_no_rows():
    c = Case(0, 64)
    r, h = c.forward()
    assert tuple(r.shape) == tuple(h.shape) == (0, 64)
    grads = c.grads(fill=3.0)
    c.backward(grads, accumulate=True)
    assert all(bool((g == 3).all()) for g in grads.values())
    dx, dy = c.backward(grads)
    assert tuple(dx.shape) == (0, 64) and not any(bool(g.any()) for g in grads.values())


def test_special_values_stay_in_their_row():
    c = Case(40, 264)
    clean = c.forward()
    gclean = c.backward(c.grads())
    c.x[3, 5], c.y[7, 200] = float("nan"), float("inf")
    keep = [i for i in range(40) if i not in (3, 7)]
    for got, want in zip((*c.forward(), *c.backward(c.grads())), (*clean, *gclean)):
        assert torch.equal(got[keep], want[keep])
    r, h = c.forward()
    assert bool(torch.isnan(r[3, 5])) and bool(torch.isnan(h[3]).all()) and bool(torch.isnan(h[7]).all())


@pytest.mark.parametrize("value", [0.0, 1e-30, 1e15])
def test_rows_of_small_and_large_values(value):
    c = Case(6, 128, stream=torch.float32)
    c.x.fill_(0.0)
    c.x[::2] = value
    c.y.mul_(value)
    c.check_forward(*c.forward())
    c.dr.mul_(0.0)
    grads = c.grads()
    c.check_backward(*c.backward(grads), grads)


def test_zero_rows_without_eps_are_nan():
    c = Case(3, 64, eps=0.0)
    c.y[1] = 0.0
    r, h = c.forward()
    assert bool(torch.isnan(r[1]).all()) and bool(torch.isnan(h[1]).all()) and bool(torch.isfinite(h[[0, 2]]).all())


def test_gradient_against_differences():
    """Along random directions, against central differences of the 64-bit forward
    pass.  The stored r carries one fp32 rounding (E of its size), which the norm
    passes on; gradients are within 2^-14 of their terms' magnitudes, the
    differences' own error (h^2 = 1e-10) is far below."""
    c = Case(48, 40, stream=torch.float32, gate=3, dr=True)
    c.y, c.dh = randn(48, 40, seed=2), randn(48, 40, seed=7, scale=1e-2)
    r, _ = c.forward()
    grads = c.grads()
    dx, dy = zc.block_norm_grad(r, dr=c.dr, dh=c.dh, y=c.y, post=c.post, gate=c.gate, residual_scale=c.scale, pre=c.pre, **grads)

    def loss(x, y, post, gate, pre):
        u = y * c.inv(y) * post * gate.repeat_interleave(16, 0)
        r = c.s32 * x + u
        return (r * c.dr.double()).sum() + (r * c.inv(r) * pre * c.dh.double()).sum()

    at = [t.double() for t in (c.x, c.y, c.post, c.gate, c.pre)]
    for i, got in enumerate((dx, dy, grads["post_grad"], grads["gate_grad"], grads["pre_grad"])):
        v = torch.randn(at[i].shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(30 + i), dtype=torch.float64)
        up, down = list(at), list(at)
        up[i], down[i] = at[i] + 1e-5 * v, at[i] - 1e-5 * v
        diff = float((loss(*up) - loss(*down)) / 2e-5)
        mine = float((got.double() * v).sum())
        slack = HALF[got.dtype] * float((got.double() * v).abs().sum()) + 2.0 ** -14 * float(got.double().norm() * v.norm())
        assert abs(mine - diff) <= slack, i


def test_same_bits_on_streams_and_in_graphs():
    c = Case(3000, 1024, gate=3)
    grads = c.grads()
    want = [*c.forward(), *c.backward(grads), *grads.values()]
    again = c.grads(fill=9.0)
    assert all(torch.equal(a, b) for a, b in zip(want, [*c.forward(), *c.backward(again), *again.values()]))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    g2 = c.grads()
    torch.cuda.synchronize()
    got = [*c.forward(stream=s), *c.backward(g2, stream=s), *g2.values()]
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    outs = dict(out=torch.empty_like(want[0]), out_norm=torch.empty_like(want[1])), dict(dx=torch.empty_like(want[2]), dy=torch.empty_like(want[3]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.forward(**outs[0])
        c.backward(g2, **outs[1])
    c.x.copy_(c.x.flip(0))
    graph.replay()
    fresh = c.grads()
    want = [*c.forward(), *c.backward(fresh), *fresh.values()]
    assert all(torch.equal(a, b) for a, b in zip(want, [*outs[0].values(), *outs[1].values(), *g2.values()]))


def test_refusals():
    c = Case(12, 64)
    g = torch.zeros(64, device="cuda")
    bad_calls = [
        lambda: zc.block_norm(c.x.half(), pre=c.pre), lambda: zc.block_norm(c.x.t(), pre=c.pre), lambda: zc.block_norm(c.x.cpu(), pre=c.pre),
        lambda: zc.block_norm(c.x), lambda: zc.block_norm(c.x, y=c.y.float(), pre=c.pre), lambda: zc.block_norm(c.x, y=c.y[:5], pre=c.pre),
        lambda: zc.block_norm(c.x, post=c.post, pre=c.pre), lambda: zc.block_norm(c.x, residual_scale=0.5, pre=c.pre),
        lambda: zc.block_norm(c.x, y=c.y, gate=torch.ones(5, 64, device="cuda")), lambda: zc.block_norm(c.x, y=c.y, gate=torch.ones(0, 64, device="cuda")),
        lambda: zc.block_norm(c.x, y=c.y, gate=torch.ones(2, 128, device="cuda")[:, :64]), lambda: zc.block_norm(c.x, y=c.y, post=c.post[:63]),
        lambda: zc.block_norm(c.x, pre=c.pre, out=torch.empty_like(c.x)), lambda: zc.block_norm(c.x, y=c.y, out_norm=torch.empty_like(c.y)),
        lambda: zc.block_norm(c.x, y=c.y, out=torch.empty(12, 64, device="cuda")), lambda: zc.block_norm(c.x, y=c.y, eps=-1.0),
        lambda: zc.block_norm(torch.zeros(2, 20000, device="cuda"), y=torch.zeros(2, 20000, device="cuda").bfloat16()),
        lambda: zc.block_norm_grad(c.x), lambda: zc.block_norm_grad(c.x, dr=c.dr, dh=c.dh), lambda: zc.block_norm_grad(c.x, dr=c.dr, pre=c.pre),
        lambda: zc.block_norm_grad(c.x, dr=c.dr.float()), lambda: zc.block_norm_grad(c.x, dr=c.dr, dy=c.y), lambda: zc.block_norm_grad(c.x, dr=c.dr, pre_grad=g),
        lambda: zc.block_norm_grad(c.x, dr=c.dr, y=c.y, gate_grad=g),
        lambda: zc.block_norm_grad(c.x, dr=c.dr, y=c.y, post=c.post, gate=c.gate, post_grad=g, gate_grad=g.bfloat16()),
        lambda: zc.block_norm_grad(c.x, dr=c.dr, dh=c.dh, pre=c.pre, pre_grad=g, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))]
    for i, call in enumerate(bad_calls):
        with pytest.raises((TypeError, ValueError, zc.DpredError)):
            call()
            pytest.fail(f"call {i} was accepted")
    assert not bool(g.any())

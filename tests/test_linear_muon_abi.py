"""The linear-layer and orthogonalised-update entry points without a GPU: what
they refuse, what they leave alone, their workspace sizes, and the algebra that
the kernels rely on.  No call here launches a kernel."""
import ctypes
import math

import numpy as np
import pytest

import zero_collectives_gb300 as zc
from zero_collectives_gb300.train import _MuonMatrix

INVAL, ALIGN, SIZE = -1, -2, -3
P = 1 << 20  # an address that is aligned to everything and never read


@pytest.fixture(scope="module")
def L():
    from zero_collectives_gb300 import build
    build.build()
    return zc.lib()


def linear(L, m=4, n=8, k=16, x=P, ldx=16, w=P, ldw=16, bdt=0, bias=None, act=0, res=None, ldr=0, pre=None, ldp=0, odt=0,
           y=P, ldy=8, ws=None, wsb=0):
    return L.dpred_linear(m, n, k, x, ldx, w, ldw, bdt, bias, act, res, ldr, pre, ldp, odt, y, ldy, ws, wsb, None)


@pytest.mark.parametrize("bad,code", [
    (dict(m=-1), INVAL), (dict(n=-5), INVAL), (dict(k=-1), INVAL), (dict(m=1 << 31), SIZE), (dict(act=4), INVAL),
    (dict(act=-1), INVAL), (dict(odt=2), INVAL), (dict(bias=P, bdt=7), INVAL), (dict(x=None), INVAL), (dict(w=None), INVAL),
    (dict(y=None), INVAL), (dict(x=P + 1), ALIGN), (dict(y=P + 2, odt=1), ALIGN), (dict(bias=P + 2, bdt=1), ALIGN),
    (dict(ldx=15), SIZE), (dict(ldw=-16), SIZE), (dict(ldy=7), SIZE), (dict(res=P, ldr=7), SIZE), (dict(pre=P + 1, ldp=8), ALIGN),
    (dict(x=P + 2), SIZE),                      # rows not 16-byte aligned: needs a workspace
    (dict(ldw=17), SIZE), (dict(x=P + 2, ws=P, wsb=64), SIZE), (dict(x=P + 2, ws=P + 8, wsb=1 << 20), ALIGN)])
def test_linear_refusals(L, bad, code):
    assert linear(L, **bad) == code
    assert L.dpred_last_error()


def test_linear_dgrad_refusals(L):
    def call(m=4, n=8, k=16, dy=P, lddy=8, w=P, ldw=16, act=0, pre=None, ldp=0, res=None, ldr=0, odt=0, dx=P, lddx=16):
        return L.dpred_linear_dgrad(m, n, k, dy, lddy, w, ldw, act, pre, ldp, res, ldr, odt, dx, lddx, None, 0, None)
    for bad, code in ((dict(m=-1), INVAL), (dict(act=9), INVAL), (dict(act=2), INVAL), (dict(act=1, pre=P, ldp=15), SIZE),
                      (dict(lddy=7), SIZE), (dict(dx=None), INVAL), (dict(res=P + 1, ldr=16), ALIGN), (dict(odt=3), INVAL),
                      (dict(dy=P + 4), SIZE)):
        assert call(**bad) == code, bad
    assert call(m=0) == 0 and call(k=0) == 0


def test_linear_wgrad_refusals(L):
    def call(m=4, n=8, k=16, dy=P, lddy=8, x=P, ldx=16, acc=0, odt=0, dw=P, lddw=16, db=None):
        return L.dpred_linear_wgrad(m, n, k, dy, lddy, x, ldx, acc, odt, dw, lddw, db, None, 0, None)
    for bad, code in ((dict(n=-1), INVAL), (dict(odt=-1), INVAL), (dict(dy=None), INVAL), (dict(x=P + 1), ALIGN),
                      (dict(lddw=15), SIZE), (dict(db=P + 2), ALIGN), (dict(dw=P + 2, odt=1), ALIGN), (dict(ldx=24 + 1), SIZE)):
        assert call(**bad) == code, bad
    assert call(n=0) == 0


def test_linear_empty_calls_need_nothing(L):
    assert linear(L, m=0, x=None, y=None) == 0
    assert linear(L, n=0, w=None, y=None) == 0


def test_linear_workspace(L):
    f = L.dpred_linear_workspace_bytes
    assert f(P, 10, 16, 16, P, 20, 16, 24) == 0
    assert f(P, 10, 17, 17, P, 20, 16, 16) == (10 * 24 * 2 + 255) // 256 * 256
    assert f(P + 2, 1, 16, 16, P, 20, 16, 17) == 256 + (20 * 16 * 2 + 255) // 256 * 256
    assert f(P, 1, 17, 17, P, 1, 17, 17) == 0  # single rows have no stride
    assert f(P, 0, 16, 16, P, 20, 17, 17) == 0


def mats(**kw):
    d = dict(rows=4, cols=6, weight=P, ldw=6, momentum=P, ldm=6, grad=P, ldg=6, scale=1.0, reserved=0)
    d.update(kw)
    t = (_MuonMatrix * 1)()
    for k, v in d.items():
        setattr(t[0], k, v)
    return t


def muon(L, table, n=1, wdt=1, gdt=0, lr=0.1, mu=0.9, wd=0.0, steps=5, coeffs=None, eps=1e-7):
    return L.dpred_muon_step(table, n, wdt, gdt, lr, mu, 1, wd, steps, coeffs, eps, None, 0, None)


@pytest.mark.parametrize("bad,code", [
    (dict(rows=-1), INVAL), (dict(rows=1 << 21), SIZE), (dict(rows=70000, cols=70000, ldw=70000, ldm=70000, ldg=70000), SIZE),
    (dict(weight=None), INVAL), (dict(momentum=P + 2), ALIGN), (dict(grad=P + 1), ALIGN), (dict(ldw=5), SIZE), (dict(ldm=0), SIZE),
    (dict(scale=float("nan")), INVAL), (dict(reserved=1), INVAL),
    (dict(rows=300, cols=300, ldw=300, ldm=300, ldg=300), SIZE)])  # no workspace
def test_muon_refuses_matrices(L, bad, code):
    assert muon(L, mats(**bad)) == code


@pytest.mark.parametrize("bad", [dict(n=-1), dict(wdt=2), dict(gdt=-1), dict(lr=float("inf")), dict(mu=float("nan")),
                                 dict(wd=float("nan")), dict(steps=0), dict(steps=33), dict(eps=-1.0),
                                 dict(coeffs=(ctypes.c_float * 3)(1.0, float("inf"), 0.0))])
def test_muon_refuses_parameters(L, bad):
    assert muon(L, mats(), **bad) == INVAL
    assert L.dpred_muon_step(None, 1, 1, 0, 0.1, 0.9, 1, 0.0, 5, None, 1e-7, None, 0, None) == INVAL


def test_newton_schulz_refusals_and_sizes(L):
    def call(batch=2, rows=300, cols=400, idt=0, src=P, ld=400, bs=120000, odt=0, out=P, ldo=400, obs=120000, ws=None, wsb=0):
        return L.dpred_newton_schulz(batch, rows, cols, idt, src, ld, bs, odt, out, ldo, obs, 5, None, 1e-7, ws, wsb, None)
    need = L.dpred_newton_schulz_workspace_bytes(2, 300, 400)
    assert need > 0 and need == L.dpred_newton_schulz_workspace_bytes(2, 400, 300)
    for bad, code in ((dict(batch=-1), INVAL), (dict(idt=5), INVAL), (dict(src=None), INVAL), (dict(ld=399), SIZE),
                      (dict(obs=10), SIZE), (dict(bs=-1), SIZE), ({}, SIZE), (dict(ws=P, wsb=need - 1), SIZE),
                      (dict(ws=P + 16, wsb=need), ALIGN)):
        assert call(**bad) == code, bad
    assert call(batch=0) == 0 and call(rows=0) == 0
    assert L.dpred_newton_schulz_workspace_bytes(5, 128, 2048) == 0      # held on chip
    assert L.dpred_newton_schulz_workspace_bytes(5, 129, 2048) > 0
    assert L.dpred_newton_schulz_workspace_bytes(0, 300, 400) == 0
    # more matrices than one launch takes reuse its workspace
    assert L.dpred_newton_schulz_workspace_bytes(640, 300, 400) == L.dpred_newton_schulz_workspace_bytes(64, 300, 400)


def test_muon_workspace_depends_on_shapes_only(L):
    a, b = mats(rows=300, cols=500), mats(rows=500, cols=300, weight=None)
    assert L.dpred_muon_workspace_bytes(a, 1) == L.dpred_muon_workspace_bytes(b, 1) > 0
    assert L.dpred_muon_workspace_bytes(mats(), 1) == 0 and L.dpred_muon_workspace_bytes(None, 3) == 0


def test_update_scale():
    assert zc.update_scale(100, 400, "spectral") == 1.0
    assert zc.update_scale(400, 100, "spectral") == 2.0
    assert zc.update_scale(400, 100, "rms") == pytest.approx(4.0)
    assert zc.update_scale(3, 5, 0.25) == 0.25


def test_split_products_and_double_steps():
    """With symmetric matrices split into diagonal and off-diagonal, the products
    that the kernels form are the full ones; and two steps worked out from one
    Gram matrix are two plain steps."""
    a, b, c = 3.4445, -4.7750, 2.0315
    rng = np.random.default_rng(3)
    x = rng.standard_normal((20, 60))
    x /= np.linalg.norm(x)

    def split(m):
        return np.diag(m).copy(), m - np.diag(np.diag(m))

    def mul(p, q):
        (d1, e1), (d2, e2) = p, q
        return np.diag(d1 * d2) + d1[:, None] * e2 + e1 * d2[None, :] + e1 @ e2

    def poly(s):
        d, e = s
        sq = e @ e
        off = (b + c * (d[:, None] + d[None, :])) * e + c * sq
        return off - np.diag(np.diag(off)) + np.diag(a + b * d + c * (d * d + np.diag(sq)))

    A = split(x @ x.T)
    full = x @ x.T
    assert np.allclose(mul(A, A), full @ full, atol=1e-14)
    assert np.allclose(poly(A), a * np.eye(20) + b * full + c * full @ full, atol=1e-13)
    y = x
    for _ in range(2):
        g = y @ y.T
        y = a * y + (b * g + c * g @ g) @ y
    p = split(poly(A))
    t = split(mul(p, A))
    a2 = split(mul(p, t))
    q = mul(split(poly(a2)), p)
    assert np.allclose(q, q.T, atol=1e-12) and np.allclose(q @ x, y, atol=1e-12)
    assert math.isclose(np.linalg.norm(y), np.linalg.norm(q @ x))

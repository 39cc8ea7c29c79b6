"""The embedding, block-norm and gradient-norm entry points without a GPU: what
they refuse, what they leave alone, and their workspace sizes.  No call here
launches a kernel."""
import ctypes

import numpy as np
import pytest

import zero_collectives_gb300 as zc
from zero_collectives_gb300.layers import _GradTensor

INVAL, ALIGN, SIZE = -1, -2, -3
P = 1 << 20  # an address that is aligned to everything and never read
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def L():
    from zero_collectives_gb300 import build
    build.build()
    return zc.lib()


def embedding(L, t=4, v=10, d=16, ib=8, ids=P, wdt=0, w=P, ldw=16, scale=1.0, odt=0, y=P, ldy=16):
    return L.dpred_embedding(t, v, d, ib, ids, wdt, w, ldw, scale, odt, y, ldy, None)


@pytest.mark.parametrize("bad,code", [
    (dict(t=-1), INVAL), (dict(v=-1), INVAL), (dict(d=-1), INVAL), (dict(t=1 << 30), SIZE), (dict(v=1 << 30), SIZE),
    (dict(d=(1 << 20) + 1), SIZE), (dict(ib=2), INVAL), (dict(ids=None), INVAL), (dict(ids=P + 4), ALIGN), (dict(ib=4, ids=P + 2), ALIGN),
    (dict(wdt=2), INVAL), (dict(odt=-1), INVAL), (dict(w=None), INVAL), (dict(y=None), INVAL), (dict(w=P + 1), ALIGN),
    (dict(y=P + 2, odt=1), ALIGN), (dict(ldw=15), SIZE), (dict(ldy=-16), SIZE), (dict(scale=NAN), INVAL), (dict(scale=INF), INVAL)])
def test_embedding_refusals(L, bad, code):
    assert embedding(L, **bad) == code and L.dpred_last_error()


def test_embedding_of_nothing(L):
    assert embedding(L, t=0, ids=None, y=None) == 0 and embedding(L, d=0, w=None, y=None) == 0


def embedding_grad(L, t=4, v=10, d=16, ib=4, ids=P, padding=-1, gdt=0, dy=P, lddy=16, scale=1.0, acc=0, odt=1, dw=P, lddw=16, ws=P,
                   wsb=1 << 30):
    return L.dpred_embedding_grad(t, v, d, ib, ids, padding, gdt, dy, lddy, scale, acc, odt, dw, lddw, ws, wsb, None)


@pytest.mark.parametrize("bad,code", [
    (dict(t=-1), INVAL), (dict(t=1 << 30), SIZE), (dict(d=1 << 21), SIZE), (dict(ib=1), INVAL), (dict(ids=None), INVAL), (dict(ids=P + 1), ALIGN),
    (dict(padding=-2), INVAL), (dict(padding=10), INVAL), (dict(gdt=3), INVAL), (dict(odt=2), INVAL), (dict(dy=None), INVAL),
    (dict(dw=None), INVAL), (dict(dw=P + 2), ALIGN), (dict(lddy=3), SIZE), (dict(lddw=15), SIZE), (dict(scale=-INF), INVAL),
    (dict(ws=None), SIZE), (dict(wsb=100), SIZE), (dict(ws=P + 128), ALIGN), (dict(t=(1 << 30) - 1, d=1 << 20, lddy=1 << 20, lddw=1 << 20), SIZE)])
def test_embedding_grad_refusals(L, bad, code):
    assert embedding_grad(L, **bad) == code and L.dpred_last_error()


def test_embedding_grad_of_nothing(L):
    assert embedding_grad(L, v=0, dw=None) == 0 and embedding_grad(L, d=0, dw=None) == 0
    assert embedding_grad(L, t=0, acc=1, ids=None, dy=None, ws=None, wsb=0) == 0
    f = L.dpred_embedding_grad_workspace_bytes
    assert f(4, 0, 16) == 0 and f(-1, 10, 16) == 0 and f(0, 10, 16) > 0
    assert f(1000, 10, 16) >= 2 * 4000 + 2 * 32 * 16 * 4 and f(1000, 10, 16) % 256 == 0


def block_norm(L, m=4, d=16, rdt=0, x=P, ldx=16, y=P, ldy=16, pdt=1, post=P, gdt=1, gate=P, gr=1, scale=1.0, wdt=1, pre=P, eps=1e-6, r=P, ldr=16,
               h=P, ldh=16):
    return L.dpred_block_norm(m, d, rdt, x, ldx, y, ldy, pdt, post, gdt, gate, gr, scale, wdt, pre, eps, r, ldr, h, ldh, None)


SHAPE_REFUSALS = [
    (dict(m=-1), INVAL), (dict(d=-1), INVAL), (dict(m=1 << 31), SIZE), (dict(d=16385, ldx=16385), SIZE), (dict(rdt=2), INVAL), (dict(eps=-1.0), INVAL),
    (dict(eps=NAN), INVAL), (dict(eps=INF), INVAL), (dict(scale=NAN), INVAL), (dict(y=None, pre=None), INVAL), (dict(y=None), INVAL),
    (dict(y=None, post=None, gate=None, scale=0.5), INVAL), (dict(pdt=2), INVAL), (dict(gdt=-1), INVAL), (dict(wdt=7), INVAL), (dict(post=P + 2), ALIGN),
    (dict(gate=P + 1, gdt=0), ALIGN), (dict(pre=P + 2), ALIGN), (dict(gr=0), SIZE), (dict(gr=3), SIZE), (dict(gr=-4), SIZE), (dict(ldy=15), SIZE),
    (dict(y=P + 1), ALIGN)]


@pytest.mark.parametrize("bad,code", SHAPE_REFUSALS + [
    (dict(x=None), INVAL), (dict(r=None), INVAL), (dict(h=None), INVAL), (dict(x=P + 2, rdt=1), ALIGN), (dict(ldr=1), SIZE), (dict(ldh=15), SIZE)])
def test_block_norm_refusals(L, bad, code):
    assert block_norm(L, **bad) == code and L.dpred_last_error()


def test_block_norm_of_nothing(L):
    assert block_norm(L, m=0, x=None, y=P, r=None, h=None) == 0 and block_norm(L, d=0) == 0


def block_norm_grad(L, m=4, d=16, rdt=0, r=P, ldr=16, dr=P, lddr=16, dh=P, lddh=16, y=P, ldy=16, pdt=1, post=P, gdt=1, gate=P, gr=1, scale=1.0,
                    wdt=1, pre=P, eps=1e-6, dx=P, lddx=16, dy=P, lddy=16, gradt=1, pg=P, gg=P, wg=P, acc=0, ws=P, wsb=1 << 30):
    return L.dpred_block_norm_grad(m, d, rdt, r, ldr, dr, lddr, dh, lddh, y, ldy, pdt, post, gdt, gate, gr, scale, wdt, pre, eps, dx, lddx, dy, lddy,
                                   gradt, pg, gg, wg, acc, ws, wsb, None)


@pytest.mark.parametrize("bad,code", [(b, c) for b, c in SHAPE_REFUSALS if "ldx" not in b and b != dict(y=None, pre=None)] + [
    (dict(r=None), INVAL), (dict(dh=None), INVAL), (dict(dx=None), INVAL), (dict(dy=None), INVAL), (dict(dr=P + 1), ALIGN), (dict(lddr=2), SIZE),
    (dict(lddh=15), SIZE), (dict(lddx=15), SIZE), (dict(lddy=0), SIZE), (dict(gradt=2), INVAL), (dict(pg=P + 2), ALIGN), (dict(post=None), INVAL),
    (dict(gate=None), INVAL), (dict(pre=None), INVAL), (dict(dr=None, pre=None, wg=None), INVAL), (dict(ws=None), SIZE), (dict(wsb=8), SIZE),
    (dict(ws=P + 16), ALIGN)])
def test_block_norm_grad_refusals(L, bad, code):
    assert block_norm_grad(L, **bad) == code and L.dpred_last_error()


def test_block_norm_grad_of_nothing(L):
    assert block_norm_grad(L, d=0) == 0 and block_norm_grad(L, m=0, acc=1, r=None) == 0
    assert block_norm_grad(L, m=0, pg=None, gg=None, wg=None) == 0
    f = L.dpred_block_norm_grad_workspace_bytes
    assert f(0, 16, 1) == 0 and f(4, 16, 3) == 0 and f(4, 16385, 1) == 0 and f(4, 16, -1) == 0
    assert f(100000, 1024, 0) > 0


def grads(*items):
    t = (_GradTensor * max(len(items), 1))()
    for e, kw in zip(t, items):
        d = dict(data=P, rows=4, cols=6, ld=6, dtype=0, counted=1)
        d.update(kw)
        for k, v in d.items():
            setattr(e, k, v)
    return t


def clip(L, *items, n=None, max_norm=1.0, eps=1e-6, result=P, ws=P, wsb=1 << 30):
    return L.dpred_clip_grads(grads(*items), len(items) if n is None else n, max_norm, eps, result, ws, wsb, None)


@pytest.mark.parametrize("bad,code", [
    (dict(rows=-1), INVAL), (dict(cols=-1), INVAL), (dict(rows=1 << 31), SIZE), (dict(cols=(1 << 40) + 1, ld=1 << 41), SIZE), (dict(dtype=2), INVAL),
    (dict(counted=2), INVAL), (dict(data=None), INVAL), (dict(data=P + 1), ALIGN), (dict(ld=5), SIZE), (dict(rows=1 << 30, cols=1 << 20, ld=1 << 21), SIZE)])
def test_gradients_refused(L, bad, code):
    assert clip(L, bad) == code and L.dpred_last_error()
    assert L.dpred_grad_norm(grads(bad), 1, P, P, 1 << 30, None) == code


def test_clip_refuses_parameters(L):
    for bad, code in ((dict(max_norm=-1.0), INVAL), (dict(max_norm=NAN), INVAL), (dict(max_norm=INF), INVAL), (dict(eps=-1.0), INVAL), (dict(eps=INF), INVAL),
                      (dict(result=None), INVAL), (dict(result=P + 2), ALIGN), (dict(ws=None), SIZE), (dict(wsb=16), SIZE), (dict(ws=P + 8), ALIGN),
                      (dict(n=-1), INVAL)):
        assert clip(L, {}, **bad) == code, bad
    assert L.dpred_clip_grads(None, 1, 1.0, 1e-6, P, P, 1 << 30, None) == INVAL
    assert L.dpred_grad_norm(grads({}), 1, None, P, 1 << 30, None) == INVAL and L.dpred_grad_norm(grads({}), 1, P + 1, P, 1 << 30, None) == ALIGN
    f = L.dpred_clip_workspace_bytes
    assert f(-1) == 0 and f(0) > 0 and f(768) == f(1) and f(769) == 2 * f(1)


@pytest.mark.parametrize("a,b,shared", [
    (dict(), dict(), True),
    (dict(), dict(data=P + 46), True), (dict(data=P + 46), dict(), True),                       # the last element
    (dict(ld=20), dict(data=P + 12, ld=20, cols=7), False), (dict(ld=20), dict(data=P + 10, ld=20), True),   # side by side
    (dict(ld=20), dict(data=P + 12, rows=1, cols=14), False), (dict(ld=20), dict(data=P + 12, rows=1, cols=15), True),  # a row in the gap
    (dict(data=P + 12, rows=1, cols=14), dict(ld=20), False),
    (dict(ld=20), dict(data=P + 12, ld=21), True),                                               # strides that do not say
    (dict(rows=30, ld=20), dict(rows=30, data=P + 12 + 40 * 7, ld=20), False)])
def test_shared_memory_is_refused(L, a, b, shared):
    """Every answer against the bytes themselves (but for unequal strides), by a
    call that is refused for its workspace alone otherwise."""
    def addresses(kw):
        d = dict(data=P, rows=4, cols=6, ld=6)
        d.update(kw)
        return {d["data"] + 2 * (r * d["ld"] + c) for r in range(d["rows"]) for c in range(d["cols"])}
    if not (a.get("ld", 6) != b.get("ld", 6) and "rows" not in a and "rows" not in b):
        assert bool(addresses(a) & addresses(b)) == shared
    # the norm of huge tables is refused later than sharing is; here only the sharing message counts
    rc = clip(L, a, b, {"data": P + (1 << 40), "rows": 1 << 30, "cols": 1 << 20, "ld": 1 << 21})
    assert rc == SIZE and (b"share memory" in L.dpred_last_error()) == shared


def test_struct_layout_matches_the_header():
    assert ctypes.sizeof(_GradTensor) == 40 and _GradTensor.counted.offset == 36
    assert np.dtype(np.int64).itemsize == 8

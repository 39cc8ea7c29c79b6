"""Sizes of gradients at the ends of what clipping accepts, without a GPU: every
call here is refused before anything is launched."""
import pytest

import zero_collectives_gb300 as zc
from zero_collectives_gb300.layers import _GradTensor

SIZE = -3
P = 1 << 20  # an address that is aligned to everything and never read
UNITS = (1 << 30) - 1  # of 16 KB, in one launch


@pytest.fixture(scope="module")
def L():
    from zero_collectives_gb300 import build
    build.build()
    return zc.lib()


def table(*items):
    t = (_GradTensor * len(items))()
    for e, kw in zip(t, items):
        for k, v in dict(dict(data=P, dtype=0, counted=1), **kw).items():
            setattr(e, k, v)
    return t


def refused(L, *items):
    t, n = table(*items), len(items)
    clip = L.dpred_clip_grads(t, n, 1.0, 1e-6, P, P, 1 << 30, None), L.dpred_last_error()
    norm = L.dpred_grad_norm(t, n, P, P, 1 << 30, None), L.dpred_last_error()
    return [rc == SIZE and b"too large" in why for rc, why in (clip, norm)] == [True, True]


@pytest.mark.parametrize("rows,cols", [((1 << 31) - 1, 1), ((1 << 31) - 8000, 1), ((1 << 31) - 1, 3), ((1 << 31) - 7, 255), ((1 << 31) - 1, 4096)])
def test_narrow_rows_are_counted_in_whole(L, rows, cols):
    """Rows that share units: with one unit more than a launch takes behind them."""
    per = 16384 // (2 * cols)
    units = -(-rows // per)
    rest = UNITS - units + 1
    narrow = dict(rows=rows, cols=cols, ld=cols + 1)
    assert refused(L, narrow, dict(data=P + (1 << 50), rows=rest, cols=8192, ld=8192))


@pytest.mark.parametrize("bad", [
    dict(rows=(1 << 31) - 1, cols=1 << 33, ld=1 << 33), dict(rows=1 << 24, cols=1 << 40, ld=1 << 40), dict(rows=2, cols=1, ld=(1 << 63) - 1),
    dict(rows=1 << 30, cols=5, ld=1 << 33), dict(rows=3, cols=4, ld=1 << 62)], ids=str)
def test_spans_that_no_address_reaches(L, bad):
    """Their sizes in bytes do not fit 64 bits: alone, and behind another gradient."""
    assert refused(L, bad) and refused(L, dict(data=P // 2, rows=2, cols=3, ld=3), bad)

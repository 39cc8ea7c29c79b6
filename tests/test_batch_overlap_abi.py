"""Batch strides of orthogonalised updates: which output layouts are refused.  No call here reaches a kernel:
each is either refused for its strides or, past that check, for the workspace it lacks (both DPRED_E_SIZE, told
apart by the message)."""
import numpy as np
import pytest

import zero_collectives_gb300 as zc

SIZE = -3
P = 1 << 20


@pytest.fixture(scope="module")
def L():
    from zero_collectives_gb300 import build
    build.build()
    return zc.lib()


def overlap_refused(L, batch, rows, cols, ldo, stride):
    rc = L.dpred_newton_schulz(batch, rows, cols, 0, P, cols, rows * cols, 0, P, ldo, stride, 5, None, 1e-7, None, 0, None)
    assert rc == SIZE
    message = L.dpred_last_error()
    message = message.decode() if isinstance(message, bytes) else message
    assert ("overlap" in message) != ("workspace" in message), message
    return "overlap" in message


@pytest.mark.parametrize("batch,rows,cols,ldo,stride,refused", [
    (2, 300, 400, 400, 120000, False),        # one after another
    (2, 300, 400, 400, 119999, True),
    (2, 300, 400, 400, 401, True),            # rows of one over rows of the other
    (2, 300, 400, 400, 400, True),
    (2, 300, 400, 800, 400, False),           # side by side
    (2, 300, 400, 799, 400, True),            # the second's rows reach the first's next rows
    (3, 300, 400, 1200, 400, False),
    (3, 300, 400, 1199, 400, True),
    (3, 300, 400, 1300, 450, False),
    (3, 300, 400, 1299, 450, True),
    (2, 300, 400, 500, 299 * 500 + 400, False),  # ends where the last row does
    (2, 300, 400, 500, 299 * 500 + 399, True),
    (2, 300, 400, 800, 399, True),
    (2, 300, 400, 400, 0, True),
    (2, 300, 400, 400, -120000, True),
    (2, 300, 400, 1200, 2000, False),         # columns 800 .. 1199 from the next row on
    (3, 300, 400, 1200, 2000, False),         # and 400 .. 799 two rows further
    (4, 300, 400, 1200, 2000, True),          # the fourth starts at column 0 of row 5: over the first
])
def test_output_strides(L, batch, rows, cols, ldo, stride, refused):
    assert overlap_refused(L, batch, rows, cols, ldo, stride) is refused


def test_random_layouts(L):
    """Against the set of addresses."""
    rng = np.random.default_rng(0)
    both = [0, 0]
    for _ in range(300):
        batch, rows, cols = int(rng.integers(2, 6)), int(rng.integers(129, 160)), int(rng.integers(129, 200))
        ldo = cols + int(rng.integers(0, 900))
        stride = int(rng.integers(1, 3 * ldo)) if rng.random() < 0.8 else int(rng.integers(1, 2 * rows * ldo))
        at = np.arange(batch)[:, None, None] * stride + np.arange(rows)[:, None] * ldo + np.arange(cols)
        refused = len(np.unique(at)) < at.size
        assert overlap_refused(L, batch, rows, cols, ldo, stride) is refused, (batch, rows, cols, ldo, stride)
        both[refused] += 1
    assert min(both) > 30


def test_one_matrix_has_no_batch_stride(L):
    assert not overlap_refused(L, 1, 300, 400, 400, 0)


def test_single_rows(L):
    """One row a matrix: only the columns must not meet."""
    for stride, code in ((4999, SIZE), (5000, None)):
        rc = L.dpred_newton_schulz(3, 1, 5000, 0, P, 0, 5000, 0, P, 0, stride, 5, None, 1e-7, None, 0, None)
        assert rc == SIZE
        m = L.dpred_last_error()
        m = m.decode() if isinstance(m, bytes) else m
        assert ("overlap" in m) == (code == SIZE)

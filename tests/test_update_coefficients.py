"""The iteration's coefficients: exactly three numbers."""
import pytest

from zero_collectives_gb300 import train


@pytest.mark.parametrize("bad", [(), (1.5,), (1.5, -0.5), (3.4, -4.8, 2.0, 0.1)])
def test_refused(bad):
    with pytest.raises(ValueError):
        train._coeffs(bad)


def test_taken():
    assert train._coeffs(None) is None
    assert list(train._coeffs((2, -1.5, 0.5))) == [2.0, -1.5, 0.5]
    assert list(train._coeffs(iter([2.0, -1.5, 0.5]))) == [2.0, -1.5, 0.5]

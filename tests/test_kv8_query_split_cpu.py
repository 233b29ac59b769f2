"""How a BF16 query row is split into two E4M3 rows, for every BF16 value (the rule of include/msa.h,
msa_kv8_attn, restated)."""
import numpy as np
import pytest

from tests import _kv8


def _split(row):
    """Values that the two E4M3 rows of a row stand for: largest element scaled into (224, 448]."""
    val = _kv8.e4m3_values()
    amax = np.abs(row).max()
    e = int(np.ceil(np.log2(amax / 448.0)))
    x = row / 2.0 ** e
    assert 224.0 < np.abs(x).max() <= 448.0
    hi = val[_kv8.e4m3_codes(x)]
    lo = val[_kv8.e4m3_codes(x - hi)]
    return (hi + lo) * 2.0 ** e


@pytest.mark.parametrize("mantissa", range(128, 256))
def test_split_of_every_value_below_a_rows_largest(mantissa):
    """All 8 bits down to 2^-9.8 of the largest, below that an absolute error of at most 2^-17.8 of it."""
    top = mantissa * 2.0 ** -7                                            # a row's largest element, 1 .. 2
    m, e = np.meshgrid(np.arange(128, 256), np.arange(-47, 1))
    x = (m * 2.0 ** (e - 7.0)).ravel()
    x = x[x <= top]
    row = np.concatenate([[top], x, -x])
    got = _split(row)
    err = np.abs(got - row)
    exact = np.abs(row) >= 2.0 ** -9.8 * top
    assert np.all(err[exact] == 0)
    assert np.all(err <= 2.0 ** -17.8 * top)
    assert np.all(err <= np.abs(row))


def test_the_bounds_are_reached():
    """The absolute error comes within 1 % of its bound, so that it passes 2^-18 of the largest."""
    row = np.array([225.0, 0.125 * (1 + 2.0 ** -7)])
    err = np.abs(_split(row) - row)
    assert err[1] == 2.0 ** -10 and 0.99 * 2.0 ** -17.8 < err[1] / 225.0 <= 2.0 ** -17.8

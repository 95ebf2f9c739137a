"""The definition of 4-bit rows that the tests use: every value that a row
holds, coded dims and rotary ones, is held again as it is."""

import numpy as np

from tests import _q4_ref as Q


def rows(seed, n=20):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((n, 512)) * np.exp(rng.standard_normal((n, 1)))
    return x.astype(np.float32).astype(np.float64)


def test_values_are_held_again():
    for seed in range(3):
        y = Q.unpack(Q.pack(rows(seed)))
        assert np.array_equal(Q.unpack(Q.pack(y.copy())), y)
        assert (y[:, :448] != 0).mean() > 0.5


def test_groups_of_far_sizes_are_held_again():
    x = rows(3)
    x[:, :448] *= np.repeat(2.0 ** -np.arange(28) * 4, 16)[None, :]
    y = Q.unpack(Q.pack(x.astype(np.float32).astype(np.float64)))
    again = Q.unpack(Q.pack(y.copy()))
    assert np.array_equal(again[:, 448:], y[:, 448:])
    # down to 2^-13 of the largest a group's scale has four significant bits
    assert np.array_equal(again[:, :16 * 12], y[:, :16 * 12])

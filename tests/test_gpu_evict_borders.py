"""GPU tests of the eviction's border among sums that are NaN: more of them than
may stay, beside sums of any size. NaN ranks above all sums, and among equal
ones the lower page stays."""

import math

import numpy as np
import pytest
import torch

import sparse_attention_csa_gb300 as csa
from tests import _q4_ref as Q
from tests.test_gpu_cache_evict import check, table

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def clean_error_word():
    yield
    torch.cuda.synchronize()
    assert csa.csa_device_error() == (0, 0)


@pytest.mark.parametrize("others", ["lognormal", "mixed", "infinite", "tiny"])
@pytest.mark.parametrize("nans,keep", [(2, 1), (3, 1), (3, 2), (3, 3), (300, 1), (300, 100), (300, 256),
                                       (300, 299), (300, 300), (300, 301), (599, 598), (600, 7)])
def test_more_nan_sums_than_may_stay(nans, keep, others):
    rng = np.random.default_rng(nans + keep)
    P, page = 600, 4
    mass = np.exp(2 * rng.standard_normal((3, P * page)))
    if others == "mixed":
        mass *= rng.choice([-1.0, 1.0], mass.shape)
    elif others == "infinite":
        mass[0, 5], mass[1, 7], mass[1, 40] = math.inf, -math.inf, math.inf
    elif others == "tiny":
        mass *= 1e-36
    for b in range(3):
        mass[b, rng.choice(P, nans, replace=False) * page + rng.integers(0, page)] = math.nan
    lens = [P * page] * 3
    want = check(mass, table(lens, page, P, rng), lens, page, keep)
    assert want[2].tolist() == [P - min(keep, P)] * 3


def test_nan_from_opposite_infinities():
    """Sums that become NaN, not rows that are."""
    rng = np.random.default_rng(5)
    P, page = 64, 8
    mass = 1.1 + rng.random((1, P * page))
    for p in (3, 20, 21, 50, 63):
        mass[0, p * page + 1], mass[0, p * page + 6] = math.inf, -math.inf
    for keep in (1, 2, 4, 5, 6):
        with np.errstate(invalid="ignore"):
            want = check(mass, table([P * page], page, P, rng), [P * page], page, keep)
        assert (want[0][0, [3, 20, 21, 50, 63][:keep]] != Q.EVICTED).all()

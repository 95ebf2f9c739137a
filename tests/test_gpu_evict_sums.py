"""GPU tests of the page sums that the eviction ranks by, against sums without
any rounding: the order of a page's rows decides nothing, equal sums keep the
lower page and larger sums the larger one."""

from fractions import Fraction

import numpy as np
import pytest
import torch

import sparse_attention_csa_gb300 as csa
from tests import _q4_ref as Q

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def clean_error_word():
    yield
    torch.cuda.synchronize()
    assert csa.csa_device_error() == (0, 0)


def exact_sum(rows):
    """Sum of fp32 rows as a whole number of 2^-200."""
    m, e = np.frexp(rows.astype(np.float64))
    assert (e > -170).all()
    return sum(int(a) << (int(b) + 176) for a, b in zip(m * 2.0 ** 24, e))


def check(pages, keeps, aligned=True):
    """pages [P, page] fp32 rows of one sequence, all in use."""
    P, page = pages.shape
    sums = [exact_sum(r) for r in pages]
    order = sorted(range(P), key=lambda p: (-sums[p], p))
    flat = torch.from_numpy(np.ascontiguousarray(pages, np.float32)).cuda().view(1, -1)
    if not aligned:
        wide = torch.empty((P * page + 1,), device="cuda")
        wide[1:] = flat[0]
        flat = wide[1:].view(1, -1)
    table = torch.arange(P, dtype=torch.int32)[None].cuda()
    rows = torch.tensor([P * page], dtype=torch.int32).cuda()
    for keep in keeps:
        out, freed, n = csa.csa_cache_evict(flat, table, rows, keep)
        gone = sorted(order[keep:])
        assert n.tolist() == [len(gone)] and freed[0, :len(gone)].tolist() == gone, keep
        assert (out[0, gone] == Q.EVICTED).all()
    return sums


def one_large(rng, page):
    """A row of 1 to 2 among rows near 2^-25, with all their 24 bits."""
    rows = rng.integers(2 ** 23, 2 ** 24, page) * 2.0 ** -49
    rows[0] = 1 + rng.integers(0, 2 ** 23) * 2.0 ** -23
    return rows


def spread(rng, page):
    return np.exp(2 * rng.standard_normal(page)).astype(np.float32).astype(np.float64)


def cancelling(rng, page):
    """Large rows of either sign that leave small ones."""
    rows = rng.integers(2 ** 23, 2 ** 24, page) * 2.0 ** -49
    k = page // 3
    big = rng.integers(2 ** 23, 2 ** 24, k) * 2.0 ** -20
    rows[:k], rows[k:2 * k] = big, -big
    return rows


def a_large_a_lane(rng, page):
    """Every lane of a page has rows of 1 beside its small ones."""
    rows = rng.integers(2 ** 23, 2 ** 24, page) * 2.0 ** -49
    rows[::7] = 1.0
    return rows


KINDS = [one_large, spread, cancelling, a_large_a_lane]


@pytest.mark.parametrize("kind", KINDS, ids=lambda f: f.__name__)
@pytest.mark.parametrize("page,P", [(16, 300), (64, 200), (63, 150), (128, 100), (500, 60), (4096, 24), (4095, 12)])
def test_same_rows_in_another_order_are_equal(kind, page, P):
    rng = np.random.default_rng(page)
    rows = kind(rng, page)
    pages = np.stack([rng.permutation(rows) for _ in range(P)])
    for aligned in (True, False):
        sums = check(pages, (1, P // 3, P - 1), aligned)
    assert len(set(sums)) == 1


@pytest.mark.parametrize("kind", KINDS, ids=lambda f: f.__name__)
@pytest.mark.parametrize("page,P", [(16, 300), (64, 200), (128, 100), (4096, 24)])
def test_sums_45_bits_apart_rank_as_they_are(kind, page, P):
    """Some pages equal, the others 2^-44 of the magnitudes' sum or a few of
    them apart."""
    rng = np.random.default_rng(page + 1)
    rows = kind(rng, page)
    small = int(np.argmin(np.abs(rows)))
    step = 2.0 ** (np.ceil(np.log2(np.abs(rows).sum())) - 44)
    pages = np.stack([rows] * P)
    pages[:, small] = rng.integers(0, P - P // 10, P) * step
    pages = np.stack([rng.permutation(r) for r in pages])
    assert (pages.astype(np.float32) == pages).all()
    check(pages, (1, P // 3, P // 2, P - 1))


@pytest.mark.parametrize("page", [64, 4096, 65536])
def test_any_rows(page):
    """Rows of many magnitudes: sums that 45 bits tell apart rank as they are."""
    rng = np.random.default_rng(page + 2)
    P = 40 if page < 65536 else 10
    pages = np.exp(3 * rng.standard_normal((P, page))).astype(np.float32).astype(np.float64)
    pages *= rng.choice([1.0, 1.0, 1.0, -1.0], pages.shape)
    sums = [Fraction(exact_sum(r), 2 ** 200) for r in pages]
    total = max(float(np.abs(r).sum()) for r in pages)
    gap = min(float(abs(a - b)) for i, a in enumerate(sums) for b in sums[:i])
    assert gap > total * 2.0 ** -45  # these rows, these pages
    check(pages, range(1, P))


def test_halfway_sums():
    """Sums at, just below and just above the middle between two numbers of 24
    and of 48 bits, put together in several ways."""
    one = [1.0, 2.0 ** -24, 0.0, 0.0, 0.0, 0.0, 0.0, 0.0]
    ways = [
        [1.0, 2.0 ** -24, 2.0 ** -60, 0, 0, 0, 0, 0], [2.0 ** -60, 2.0 ** -24, 1.0, 0, 0, 0, 0, 0],
        [1.0 + 2.0 ** -23, -2.0 ** -24, 2.0 ** -60, 0, 0, 0, 0, 0],
        [0, 2.0 ** -25, 2.0 ** -60, 2.0 ** -25, 0, 0, 0, 1.0], [2.0, -1.0, 2.0 ** -24, 0, 0, 0, 2.0 ** -60, 0],
    ]
    deep = [
        [1.0, 2.0 ** -30, 2.0 ** -54, 2.0 ** -62, 0, 0, 0, 0], [2.0 ** -62, 2.0 ** -54, 2.0 ** -30, 1.0, 0, 0, 0, 0],
        [1.0, 2.0 ** -30 + 2.0 ** -53, -2.0 ** -54, 2.0 ** -62, 0, 0, 0, 0],
        [2.0 ** -61, -2.0 ** -62, 1.0, 2.0 ** -54, 0, 2.0 ** -30, 0, 0],
    ]
    for same in (ways, deep):
        assert len({exact_sum(np.array(w)) for w in same}) == 1
        pages = np.array(same * 3)
        check(pages, range(1, len(pages)))
        check(-pages, range(1, len(pages)))
    down = [1.0, 2.0 ** -24, -2.0 ** -44, 0, 0, 0, 0, 0]
    up = [1.0, 2.0 ** -24, 2.0 ** -44, 0, 0, 0, 0, 0]
    check(np.array([down, one, up, one, down, up]), range(1, 6))

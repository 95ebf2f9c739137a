"""GPU tests of the eviction over pages as large as its sizes allow: what it
reads and how long it takes follow the rows in use."""

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


def run(mass, P, rows, keep, **kw):
    pages = torch.arange(7, 7 + P, dtype=torch.int32)[None].cuda()
    used = torch.tensor([rows], dtype=torch.int32).cuda()
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    csa.csa_cache_evict(mass, pages, used, keep, **kw)
    start.record()
    got = csa.csa_cache_evict(mass, pages, used, keep, **kw)
    end.record()
    torch.cuda.synchronize()
    return [x.tolist() for x in got], start.elapsed_time(end)


# 2^31 - 1 rows: one at a time, their count beside INT32_MAX
@pytest.mark.parametrize("P,page", [(1, 2 ** 31 - 1), (1, 2 ** 31 - 4), (2, 2 ** 30 - 1), (3, 2 ** 29)])
def test_few_rows_of_a_large_page(P, page):
    mass = torch.empty((1, P * page), dtype=torch.float32, device="cuda")
    mass[:, :64] = torch.rand(64)
    for rows in (1, 3, 31, 33, 64):
        (out, freed, n), ms = run(mass, P, rows, 0)
        assert out == [list(range(7, 7 + P))] and freed == [[-1] * P] and n == [0]  # it has room for more
        assert ms < 5.0  # a page's 2^26 rows a lane would take far longer


def test_large_pages_in_use():
    """Pages of 2^24 rows, the last one hardly used: the heavier ones stay."""
    page, P = 1 << 24, 5
    mass = torch.full((1, P * page), 2.0 ** -30, device="cuda")
    for p, x in enumerate((3.0, 1.0, 2.0, 1.0, 5.0)):
        mass[0, p * page + 12345 + p] = x
    (out, freed, n), _ = run(mass, P, 4 * page + 9, 3)
    e = Q.EVICTED
    assert out == [[7, e, 9, e, 11]] and freed == [[8, 10, -1, -1, -1]] and n == [2]

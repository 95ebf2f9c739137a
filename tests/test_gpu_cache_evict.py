"""GPU tests of the pages given back by the weight of their rows: equal to the
definition, number by number."""

import math

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


def table(lens, page, max_pages, rng, holes=0.0):
    t = np.full((len(lens), max_pages), -1, np.int32)
    total = sum(max(-(-n // page), 0) for n in lens)
    perm, at = rng.permutation(total + 3), 0
    for b, n in enumerate(lens):
        for p in range(max(-(-n // page), 0)):
            t[b, p] = perm[at]
            at += 1
    t[rng.random(t.shape) < holes] = -1
    t[rng.random(t.shape) < holes] = Q.EVICTED
    return t


def check(mass, pages, rows, page, keep, first=0, last=0, in_place=False):
    m = torch.from_numpy(mass.astype(np.float32)).cuda()
    p = torch.from_numpy(pages).cuda()
    r = torch.tensor(rows, dtype=torch.int32).cuda()
    out, freed, n = csa.csa_cache_evict(m, p, r, keep, keep_first=first, keep_last=last,
                                        out=p if in_place else None)
    torch.cuda.synchronize()
    want = Q.evict(mass.astype(np.float32), pages, rows, page, keep, first, last)
    for g, w, what in zip((out, freed, n), want, ("table", "freed", "n_freed")):
        assert np.array_equal(g.cpu().numpy(), w), what
    assert in_place or np.array_equal(p.cpu().numpy(), pages)
    return want


@pytest.mark.parametrize("page", [1, 3, 4, 16, 40, 64, 128, 500])
@pytest.mark.parametrize("keep,first,last", [(0, 0, 0), (1, 0, 0), (7, 0, 0), (7, 1, 1), (9, 65, 100),
                                             (3, 10 ** 9, 0), (3, 0, 2 ** 31 - 1), (10 ** 6, 0, 0)])
def test_against_definition(page, keep, first, last):
    rng = np.random.default_rng(page * 31 + keep)
    lens = [0, 1, page, page + 1, 20 * page, 20 * page - 1, 33 * page + page // 2, -4]
    P = 40
    mass = np.exp(2 * rng.standard_normal((len(lens), P * page)))
    check(mass, table(lens, page, P, rng), lens, page, keep, first, last)
    check(mass, table(lens, page, P, rng, holes=0.2), lens, page, keep, first, last, in_place=True)


@pytest.mark.parametrize("P,page", [(1023, 16), (1024, 4), (1025, 16), (5000, 16), (24576, 1), (16384, 16)])
def test_many_pages(P, page):
    rng = np.random.default_rng(P)
    lens = [P * page, P * page - page // 2, P * page // 3]
    mass = np.exp(2 * rng.standard_normal((3, P * page)))
    for keep in (1, P // 4, P - 1):
        check(mass, table(lens, page, P, rng), lens, page, keep, 64, 300)


def test_equal_sums_keep_the_lower_page():
    rng = np.random.default_rng(0)
    P, page = 1500, 8
    lens = [P * page, P * page, P * page]
    mass = np.zeros((3, P * page))
    mass[1, 0::page] = rng.integers(0, 3, P)                 # few distinct sums
    mass[2, :] = 1.0
    mass[2, 5::page] = rng.permutation(P) < 100
    for keep in (1, 400, 1499):
        check(mass, table(lens, page, P, rng), lens, page, keep, in_place=True)


def test_close_sums_beside_far_ones():
    """More sums in one bin of the interval than are ranked at once: close
    together, equal among them, beside a tiny and a huge one."""
    rng = np.random.default_rng(1)
    P, page = 3000, 4
    lens = [P * page] * 2
    mass = np.ones((2, P * page))
    mass[0] += rng.integers(0, 60, P * page) * 2.0 ** -23     # few distinct sums
    mass[1] += rng.random(P * page) * 2.0 ** -10
    mass[:, :page], mass[:, page:2 * page] = 1e-30, 1e30
    for keep in (1, 2, 700, 1500, 2999):
        check(mass, table(lens, page, P, rng), lens, page, keep)


def test_sums_of_any_kind():
    """Negative, tiny, infinite and NaN sums rank as numbers do, NaN above all."""
    rng = np.random.default_rng(2)
    P, page = 60, 4
    mass = rng.standard_normal((2, P * page)) * 1e-30
    mass[0, 17], mass[0, 50], mass[0, 90], mass[0, 130] = math.nan, math.inf, -math.inf, -1e30
    mass[1] = -np.abs(mass[1])
    mass[1, :40] = -0.0
    mass[1, 40:80] = 0.0
    for keep in (1, 2, 3, 10, 57, 59):
        check(mass, table([P * page] * 2, page, P, rng), [P * page] * 2, page, keep)


def test_unaligned_mass_and_large_batch():
    rng = np.random.default_rng(3)
    B, P, page = 700, 9, 4
    wide = torch.rand((B * P * page + 1,)).cuda()
    mass = wide[1:].view(B, P * page)
    lens = rng.integers(0, P * page + 1, B).tolist()
    t = table(lens, page, P, rng)
    out, freed, n = csa.csa_cache_evict(mass, torch.from_numpy(t).cuda(),
                                        torch.tensor(lens, dtype=torch.int32).cuda(), 4)
    want = Q.evict(mass.cpu().numpy(), t, lens, page, 4)
    for g, w in zip((out, freed, n), want):
        assert np.array_equal(g.cpu().numpy(), w)


def test_rows_beyond_the_table_are_cut_and_recorded():
    rng = np.random.default_rng(4)
    mass = rng.random((1, 32))
    t = table([32], 4, 8, rng)
    p, r = torch.from_numpy(t).cuda(), torch.tensor([1000], dtype=torch.int32).cuda()
    out, freed, n = csa.csa_cache_evict(torch.from_numpy(mass).float().cuda(), p, r, 2)
    assert csa.csa_device_error()[0] == 6
    want = Q.evict(mass.astype(np.float32), t, [32], 4, 2)
    assert np.array_equal(out.cpu().numpy(), want[0]) and n.tolist() == [6]


def test_nothing_to_do():
    e = torch.empty((0, 8), dtype=torch.int32).cuda()
    out, freed, n = csa.csa_cache_evict(torch.empty((0, 32)).cuda(), e, e[:, 0].contiguous(), 2)
    assert out.shape == (0, 8) and n.shape == (0,)
    out, freed, n = csa.csa_cache_evict(torch.empty((3, 0)).cuda(), torch.empty((3, 0), dtype=torch.int32).cuda(),
                                        torch.zeros(3, dtype=torch.int32).cuda(), 2)
    assert out.shape == (3, 0) and n.tolist() == [0, 0, 0]


def test_captured_and_replayed():
    rng = np.random.default_rng(6)
    P, page = 100, 16
    t = table([P * page] * 3, page, P, rng)
    mass = torch.rand((3, P * page)).cuda()
    p, r = torch.from_numpy(t).cuda(), torch.tensor([P * page] * 3, dtype=torch.int32).cuda()
    out, freed, n = torch.empty_like(p), torch.empty_like(p), torch.empty_like(r)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=torch.cuda.Stream()):
        csa.csa_cache_evict(mass, p, r, 30, out=out, freed=freed, n_freed=n)
    for seed in range(3):
        mass.copy_(torch.rand((3, P * page), generator=torch.Generator().manual_seed(seed)))
        g.replay()
        torch.cuda.synchronize()
        want = Q.evict(mass.cpu().numpy(), t, [P * page] * 3, page, 30)
        for a, w in zip((out, freed, n), want):
            assert np.array_equal(a.cpu().numpy(), w)

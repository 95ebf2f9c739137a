"""GPU tests of the paged indexer with scores that are not finite: which rows
it takes, and that it writes nothing beside them."""

import math

import numpy as np
import pytest
import torch

import sparse_attention_csa_gb300 as csa
from tests import _paged_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def clean_error_word():
    yield
    torch.cuda.synchronize()
    assert csa.csa_device_error() == (0, 0)


def i32(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32)).cuda()


def ranked(q, cache, w, table, pos, ratio, topk):
    """Rows and scores of the formula when a product or a score is not finite:
    a product that is NaN counts as 0 (max(0, .) keeps what is above 0), a score
    that is NaN ranks above all others, ties to the lower row."""
    page = cache.shape[1]
    idx, val = np.full((len(pos), topk), -1, np.int64), np.full((len(pos), topk), -np.inf)
    for t, p in enumerate(pos):
        n = (p + 1) // ratio
        _, k = R.gather(cache, table, page, 0, range(n))
        with np.errstate(invalid="ignore"):
            dots = k @ R.f64(q[t]).T
            s = np.where(dots > 0, dots, 0.0) @ R.f64(w[t])
            best = np.sort(np.lexsort((np.arange(n), -s, ~np.isnan(s)))[:topk])
        idx[t, :len(best)], val[t, :len(best)] = best, s[best]
    return idx, val


def check(q, cache, w, table, pos, ratio, topk):
    """Rows and values as in the formula; what lies behind the outputs stays."""
    T = len(pos)
    more = 200000  # int32 and fp32 entries behind the outputs
    out = torch.full((T * topk + more,), -77, dtype=torch.int32, device="cuda")
    val = torch.full((T * topk + more,), -77.0, device="cuda")
    csa.csa_indexer_topk_paged(q, cache, w, i32(table), i32([0] * T), i32(pos), ratio, topk, return_value=True,
                               out=out[:T * topk].view(T, topk), out_val=val[:T * topk].view(T, topk))
    want, wval = ranked(q, cache, w, table, pos, ratio, topk)
    assert np.array_equal(out[:T * topk].view(T, topk).cpu().numpy(), want)
    assert np.array_equal(R.f64(val[:T * topk].view(T, topk)), wval, equal_nan=True)
    assert (out[T * topk:] == -77).all() and (val[T * topk:] == -77).all()


@pytest.mark.parametrize("n,topk", [(300, 40), (9000, 512), (70000, 512), (70000, 20)])
@pytest.mark.parametrize("what", ["inf key", "nan key", "inf weight", "-inf weight", "nan weight", "both"])
def test_indexer_scores_that_are_not_finite(n, topk, what):
    """Few or many of them, over one CTA's rows or a cluster's."""
    gen = torch.Generator().manual_seed(n)
    ratio, H, D = 2, 8, 64
    table, total = R.pool_rows([n], 64, seed=1)
    cache = R.grid(gen, (total, 64, D), 1.0, torch.bfloat16).cuda()
    q = R.grid(gen, (2, H, D), 1.0, torch.bfloat16).cuda()
    w = R.grid(gen, (2, H), 0.25, torch.float32).cuda()
    rows = np.random.default_rng(n).choice(n, 30, replace=False)
    for i, r in enumerate(rows):
        page, at = R.slot(table, 64, 0, r)
        if what in ("inf key", "both"):
            cache[page, at, i] = math.inf if i % 2 else -math.inf
        if what == "nan key":
            cache[page, at, i] = math.nan
    if "weight" in what or what == "both":
        w[0, 3] = {"inf weight": math.inf, "-inf weight": -math.inf, "both": math.inf}.get(what, math.nan)
        w[1, 0] = math.inf if what == "both" else w[1, 0]
        w[1, 5] = -math.inf if what == "both" else w[1, 5]
    pos = [2 * n - 1, n]
    check(q, cache, w, table, pos, ratio, topk)


@pytest.mark.parametrize("topk", [150, 2000])
@pytest.mark.parametrize("n", [3000, 12000, 70000])
@pytest.mark.parametrize("share", [0.0005, 0.1, 0.6])
def test_nan_scores_among_negative_ones(n, topk, share):
    """Rows of two infinite products that cancel (a NaN score) among finite
    scores, most of them negative: the border is negative too where many rows
    are taken, or only NaN are taken."""
    gen = torch.Generator().manual_seed(n)
    table, total = R.pool_rows([n], 64, seed=1)
    cache = R.grid(gen, (total, 64, 64), 0.5, torch.bfloat16).cuda()
    q = R.grid(gen, (3, 8, 64), 0.5, torch.bfloat16).cuda()
    w = -(R.grid(gen, (3, 8), 0.125, torch.float32).abs() + 0.125).cuda()
    q[:, :2, 5], w[:, 0] = 1.0, 0.125
    rng = np.random.default_rng(n)
    rows = rng.choice(n, max(1, int(share * n)), replace=False)
    at = torch.from_numpy(np.array([R.slot(table, 64, 0, r) for r in rows])).cuda()
    cache[at[:, 0], at[:, 1], 5] = math.inf
    pos = [4 * n - 1, 2 * n, 4 * n - 400]
    check(q, cache, w, table, pos, 4, topk)

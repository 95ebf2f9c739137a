"""GPU tests of the paged attention and the paged indexer with values that are
not finite: what they do to a token that sees them, and to no other."""

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


class Window:
    """Tokens over one sequence's window rows: `n` keys each, one a token."""

    def __init__(self, n, tokens, H=6, sinks=None, seed=0):
        gen = torch.Generator().manual_seed(seed)
        self.table, total = R.pool_rows([4 * n], 64, seed=seed)
        self.ori = torch.randn((total, 64, 512), generator=gen).bfloat16().cuda()
        self.q = torch.randn((tokens, H, 512), generator=gen).bfloat16().cuda()
        self.pos = [(4 * n - 1 - 3 * t) % (4 * n) for t in range(tokens)]
        self.n, self.sinks = n, None if sinks is None else torch.tensor(sinks, dtype=torch.float32).cuda()

    def check(self):
        """The same entries NaN as in the formula, the others within its bounds."""
        T = len(self.pos)
        out, lse = csa.csa_sparse_mla_paged(self.q, self.ori, None, None, i32(self.table), None, i32([0] * T),
                                            i32(self.pos), self.sinks, R.inv_sqrt(512), 1, self.n - 1,
                                            return_softmax_lse=True)
        with np.errstate(invalid="ignore"):
            want, wlse, tol, ltol = R.attention(self.q, self.ori, None, None, self.table, None, [0] * T,
                                                self.pos, self.sinks, R.inv_sqrt(512), 1, self.n - 1)
        for got, w, t in ((R.f64(out), want, tol), (R.f64(lse), wlse, ltol)):
            nan = np.isnan(w)
            assert np.array_equal(np.isnan(got), nan)
            assert (np.abs(got - w)[~nan] <= t[~nan]).all()
        return want


# keys of a token in one tile; in one CTA's two; in parts that are joined
@pytest.mark.parametrize("n,tokens", [(40, 3), (100, 160), (100, 400), (3000, 4)])
@pytest.mark.parametrize("sinks", [None, [0.5, -math.inf, -1.0, 3.0, 0.0, 1.0]])
def test_nan_query(n, tokens, sinks):
    """A head of a token whose query holds a NaN is NaN; its neighbours are not."""
    c = Window(n, tokens, sinks=sinks)
    c.q[0, 1, 17] = math.nan
    c.q[1, 0] = math.nan
    want = c.check()
    assert np.isnan(want[0, 1]).all() and not np.isnan(want[0, 0]).any()


@pytest.mark.parametrize("n,tokens", [(40, 3), (100, 400), (3000, 4)])
def test_nan_key(n, tokens):
    """A key with a NaN, seen by some tokens only."""
    c = Window(n, tokens)
    seen = [c.pos[0] - 1, c.pos[-1]]
    for r in seen:
        page, at = R.slot(c.table, 64, 0, r)
        c.ori[page, at, 100] = math.nan
    want = c.check()
    assert np.isnan(want[0]).all() and np.isnan(want[-1]).all()
    assert tokens < 10 or not np.isnan(want).all()


@pytest.mark.parametrize("n,tokens", [(40, 3), (100, 400), (3000, 4)])
def test_sinks_that_are_not_finite(n, tokens):
    """NaN and +inf have no softmax: NaN, as in the formula; -inf is no sink."""
    want = Window(n, tokens, sinks=[math.nan, 0.0, math.inf, -math.inf, 1.0, 300.0]).check()
    assert np.isnan(want[:, [0, 2]]).all() and not np.isnan(want[:, [1, 3, 4, 5]]).any()
